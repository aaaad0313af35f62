"""Measured cases of the operators around rotary positions and chunked prompts: the rotation of Q and K (with its
gradient), the 8-bit cache's append with the rotation on the way, and attention of chunks of new tokens over that cache.

`run` computes a case in elementary torch operations when `own` is false, and through the library's entry points when
it is true. `exact` computes the same outputs from the definitions in 64 bits.
"""
import math
import random

import torch

own = False

BLOCK = 64          # tokens per cache block: one scale per block and KV head


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decoding step of a batch: Q and K of one token per sequence, latency counts
        dict(name="rope_step", op="rope", b=1, t=64, hq=64, hkv=8, d=128, rot=128, axes=1, interleaved=False, bf16=True,
             inverse=False, batched=False),
        # a training step's Q and K on their way from the projections to the attention's layout
        dict(name="rope_train", op="rope", b=2, t=8192, hq=16, hkv=16, d=128, rot=128, axes=1, interleaved=False, bf16=True,
             inverse=False, batched=True),
        # the gradient on patches of a video (time, height, width), fp32, half of each head rotated, pairs side by side
        dict(name="rope_video_grad", op="rope", b=1, t=11111, hq=12, hkv=4, d=96, rot=48, axes=3, interleaved=True, bf16=False,
             inverse=True, batched=False),
        # one decoding step of a batch: one token rotated and appended to each sequence
        dict(name="append_step", op="append", seqs=64, tokens=64, past=2000, hkv=8, d=128, rot=128, axes=1, interleaved=False),
        # prompts rotated and written to the cache, most of them behind tokens that are there
        dict(name="append_prompts", op="append", seqs=9, tokens=30011, past=500, hkv=8, d=128, rot=128, axes=1,
             interleaved=False),
        # images among text: three axes, smaller heads
        dict(name="append_video", op="append", seqs=5, tokens=9001, past=77, hkv=4, d=80, rot=80, axes=3, interleaved=True),
        # one user's follow-up question after a short chat: latency
        dict(name="chunk_short", op="chunk", seqs=1, tokens=19, past=300, hq=32, hkv=8, d=128),
        # a step that carries one piece of a prompt and decoding sequences, one token each
        dict(name="chunk_mixed", op="chunk", seqs=25, tokens=1048, past=8192, hq=64, hkv=8, d=128, ones=True),
        # several prompts' next pieces, smaller heads
        dict(name="chunk_batch", op="chunk", seqs=7, tokens=9000, past=6000, hq=16, hkv=4, d=64),
        # a piece of a long prompt: 4096 tokens at the end of 32768
        dict(name="chunk_prefill", op="chunk", seqs=1, tokens=4096, past=28672, hq=32, hkv=8, d=128),
        # a few lines asked about long documents: few rows, the length has to be split
        dict(name="chunk_long", op="chunk", seqs=2, tokens=130, past=131072, hq=64, hkv=8, d=128),
        # wide heads without groups
        dict(name="chunk_wide", op="chunk", seqs=4, tokens=3000, past=5000, hq=16, hkv=16, d=256),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, evenly over the logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["rope", "append", "chunk", "chunk"])
    interleaved, axes = rng.random() < 0.4, rng.choice([1, 1, 2, 3])
    if op == "rope":
        hq, hkv = rng.choice([(64, 8), (16, 16), (32, 8), (12, 4), (6, 1), (7, 7)])
        d = rng.choice([64, 128, 256, 80, 96, 40])
        return dict(op=op, b=1, t=_log(rng, 1, 16000 * 1024 // ((hq + hkv) * d)), hq=hq, hkv=hkv, d=d,
                    rot=d if rng.random() < 0.7 else d // 16 * 8, axes=axes, interleaved=interleaved,
                    bf16=rng.random() < 0.7, inverse=rng.random() < 0.4, batched=rng.random() < 0.5)
    if op == "append":
        seqs, d = _log(rng, 1, 96), rng.choice([64, 128, 256, 80, 112, 192])
        tokens = seqs if rng.random() < 0.4 else _log(rng, seqs, 28000 * 128 // max(d, 128))
        return dict(op=op, seqs=seqs, tokens=tokens, past=_log(rng, 1, 1500), hkv=rng.choice([1, 2, 5, 8]), d=d,
                    rot=d if rng.random() < 0.7 else d // 16 * 8, axes=axes, interleaved=interleaved)
    hq, hkv = rng.choice([(32, 8), (64, 8), (16, 16), (8, 1), (12, 4), (20, 2), (7, 7)])
    seqs, d = _log(rng, 1, 32), rng.choice([64, 128, 128, 256, 80, 48, 192])
    tokens = _log(rng, seqs, 5000)
    # no more to read, or to multiply, than the largest listed case has
    past = _log(rng, 1, min(40000, 180000000 // (seqs * hkv * d), 300000000000 // (hq * d * tokens)))
    return dict(op=op, seqs=seqs, tokens=tokens, past=past, hq=hq, hkv=hkv, d=d, ones=rng.random() < 0.3)


def _lengths(case):
    """The sequences' new tokens: the case's own, whatever the seed, at least one each. `ones`: all but the first have
    one."""
    n, total = case["seqs"], case["tokens"]
    if case.get("ones"):
        return [total - (n - 1)] + [1] * (n - 1)
    rng = random.Random("%s %s %s" % (case["op"], n, total))
    share = [rng.random() ** 2 + 0.02 for _ in range(n)]
    lens = [1 + int((total - n) * x / sum(share)) for x in share]
    lens[share.index(max(share))] += total - sum(lens)
    return lens


def _past(case):
    """Tokens held before. An append: none for the first sequence of several, up to `past` for the others. A chunk:
    between a quarter of `past` and `past`, which the first one has."""
    rng = random.Random("past %s %s" % (case["seqs"], case["past"]))
    if case["op"] == "append":
        return [0 if i == 0 and case["seqs"] > 1 else rng.randint(1, case["past"]) for i in range(case["seqs"])]
    return [case["past"]] + [rng.randint(case["past"] // 4, case["past"]) for _ in range(case["seqs"] - 1)]


def work(case):
    d = case["d"]
    if case["op"] == "rope":
        values = float(case["b"] * case["t"] * (case["hq"] + case["hkv"]) * d)
        return {"bytes": values * 2 * (2 if case["bf16"] else 4) + 4.0 * case["axes"] * case["t"], "flops": 3.0 * values}
    lens, hkv = _lengths(case), case["hkv"]
    if case["op"] == "append":
        total = float(sum(lens) * hkv)
        return {"bytes": 2.0 * total * d * (2 + 1) + 4.0 * case["axes"] * sum(lens), "flops": 3.0 * total * d}
    hq, past = case["hq"], _past(case)
    held = sum(lens) + sum(past)
    pairs = sum(n * p + n * (n + 1) / 2 for n, p in zip(lens, past))
    return {"bytes": 2.0 * held * hkv * d + sum(lens) * hq * (4.0 * d + 4) + 8.0 * hkv * sum(-(-(n + p) // BLOCK)
                                                                                       for n, p in zip(lens, past)),
            "flops": 4.0 * hq * d * pairs}


# ------------------------------------------------------------------ inputs
def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _cumulative(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return _ints(at)


def _frequencies(case):
    """Radians per position of each pair, falling from 1, and the axis that each goes by: neighbouring thirds (halves) of
    the pairs."""
    n = case["rot"] // 2
    return [1e4 ** (-i / n) for i in range(n)], [i * case["axes"] // n for i in range(n)]


def _rope(case):
    """The frequencies as 64 bits hold them, for the formulas, and as parts of a turn in units of 2^-64, for the call."""
    freq, axis = _frequencies(case)
    turns = [int(round(f / (2 * math.pi) * 2 ** 64)) for f in freq]
    turns = [x - 2 ** 64 if x >= 2 ** 63 else x for x in turns]
    return dict(turns=torch.tensor(turns, dtype=torch.int64, device="cuda"), axis=_ints(axis),
                interleaved=case["interleaved"]), torch.tensor(freq, dtype=torch.float64, device="cuda")


def _positions(gen, case, t):
    """[axes, t]: text behind one another, from far on; patches of frames of 13 x 17 where there are several axes."""
    at = torch.arange(t, device="cuda")
    start = torch.randint(0, 1 << 20, (1,), generator=gen, device="cuda")
    if case["axes"] == 1:
        return (at + start).to(torch.int32)[None]
    parts = [at // 221 + start, at // 17 % 13 + 3, at % 17 - 8]
    return torch.stack(parts[: case["axes"]]).to(torch.int32)


def _cache(gen, blocks, hkv, d):
    """A pool in use: codes of normal values (K and V of magnitude about 1), scales powers of two that differ by block
    and head."""
    codes = []
    for _ in range(2):
        x = torch.empty(blocks, hkv, BLOCK, d, dtype=torch.uint8, device="cuda")
        for i in range(0, blocks, 512):
            j = min(blocks, i + 512)
            x[i:j] = (_randn(gen, j - i, hkv, BLOCK, d) * 48).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        codes.append(x)
    scales = [torch.exp2(torch.randint(-7, -4, (blocks, hkv), generator=gen, device="cuda").float()) for _ in range(2)]
    return dict(k=codes[0], v=codes[1], k_scale=scales[0], v_scale=scales[1])


def _table(gen, lens, spare):
    """Block table over a pool of shuffled blocks, and the pool's size; `spare` more blocks for each sequence."""
    width = max(-(-n // BLOCK) for n in lens) + spare
    blocks = len(lens) * width + 3
    perm = torch.randperm(blocks, generator=gen, device="cuda")[: len(lens) * width]
    return perm.to(torch.int32).view(len(lens), width).contiguous(), blocks


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    d, s = case["d"], dict(case=case)
    if case["op"] == "rope":
        s["rope"], s["freq"] = _rope(case)
        s["positions"] = _positions(gen, case, case["t"])
        dtype = torch.bfloat16 if case["bf16"] else torch.float32
        for name, heads in (("q", case["hq"]), ("k", case["hkv"])):
            # a projection's output, [batch, token, head, d] in memory
            s[name] = _randn(gen, case["b"], case["t"], heads, d).to(dtype).transpose(1, 2)
            s[name] = s[name] if case["batched"] else s[name][0]
        return s
    lens, past, hkv = _lengths(case), _past(case), case["hkv"]
    s.update(lens=lens, cu=_cumulative(lens))
    s["table"], blocks = _table(gen, [a + b for a, b in zip(past, lens)], 1 if case["op"] == "chunk" else 0)
    s["cache"] = _cache(gen, blocks, hkv, d)
    if case["op"] == "append":
        s["rope"], s["freq"] = _rope(case)
        s["positions"] = _positions(gen, case, sum(lens))
        # a token now and then is larger than what its block holds, and the block's scale has to grow
        s["k"], s["v"] = (_randn(gen, sum(lens), hkv, d).mul_(4).to(torch.bfloat16).transpose(0, 1) for _ in range(2))
        s["start"] = _ints(past)
        return s
    s["q"] = _randn(gen, sum(lens), case["hq"], d).to(torch.bfloat16).transpose(0, 1)
    s["lengths"] = _ints([a + b for a, b in zip(past, lens)])
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return _OWN[op](state)
    return _PLAIN[op](state)


def _pools(c):
    """The cache as outputs: codes as the e4m3 values they are, and their scales."""
    return dict(k=c["k"].view(torch.float8_e4m3fn), v=c["v"].view(torch.float8_e4m3fn), k_scale=c["k_scale"],
                v_scale=c["v_scale"])


def _own_rope(s):
    import exact_attention_79_gb300 as fa
    out = [None, None]
    if s["case"]["batched"]:                      # to the layout that attention wants, [batch, head, token, d] in memory
        out = [torch.empty(s[x].shape, dtype=s[x].dtype, device=s[x].device) for x in ("q", "k")]
    q, k = fa.rope(s["q"], s["k"], fa.Rope(**s["rope"]), s["positions"], inverse=s["case"]["inverse"], q_out=out[0],
                   k_out=out[1])
    return dict(q=q, k=k)


def _own_append(s):
    import exact_attention_79_gb300 as fa
    fa.cache8_append(fa.Cache8(**s["cache"]), s["k"], s["v"], s["cu"], s["table"], s["start"], rope=fa.Rope(**s["rope"]),
                     positions=s["positions"])
    return _pools(s["cache"])


def _own_chunk(s):
    import exact_attention_79_gb300 as fa
    o, lse = fa.fwd_cache8_packed(s["q"], fa.Cache8(**s["cache"]), s["cu"], s["table"], s["lengths"], causal=True)
    return dict(o=o, lse=lse)


_OWN = dict(rope=_own_rope, append=_own_append, chunk=_own_chunk)


# ---- plain forms
def _angles(s, sign):
    """cos and sin [t, pairs] in fp32, from angles in 64 bits: 32 lose the far positions' angles."""
    t = s["positions"].double()[s["rope"]["axis"].long()].t() * s["freq"] * sign
    return t.cos().float(), t.sin().float()


def _rotated(x, cos, sin, interleaved):
    """x [..., t, d] in 32 bits (or 64), its first 2 * pairs columns rotated."""
    n = cos.shape[-1]
    first, second = (x[..., : 2 * n : 2], x[..., 1 : 2 * n : 2]) if interleaved else (x[..., :n], x[..., n : 2 * n])
    a, b = first * cos - second * sin, first * sin + second * cos
    turned = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([turned, x[..., 2 * n :]], -1)


def _plain_rope(s):
    cos, sin = _angles(s, -1.0 if s["case"]["inverse"] else 1.0)
    out = {}
    for name in ("q", "k"):
        y = _rotated(s[name].float(), cos, sin, s["case"]["interleaved"]).to(s[name].dtype)
        out[name] = y.contiguous() if s["case"]["batched"] else torch.empty_like(s[name]).copy_(y)
    return out


def _power_scale(amax):
    """The smallest power of two s with amax / s <= 448 (at least 2^-126), 1 where amax is 0. amax = m 2^e, m in
    [1/2, 1); 448 = 7/8 2^9."""
    m, e = torch.frexp(amax)
    return torch.where(amax > 0, torch.exp2((e - 9 + (m > 0.875).int()).clamp_min(-126).float()), torch.ones_like(amax))


def _codes(x):
    return x.to(torch.float8_e4m3fn).view(torch.uint8)


def _plain_append(s):
    c = s["cache"]
    cu, start, table = s["cu"].long(), s["start"].long(), s["table"].long()
    token = torch.arange(s["k"].shape[1], device=cu.device)
    seq = torch.searchsorted(cu, token, right=True) - 1
    at = start[seq] + token - cu[seq]
    block, slot = table[seq, at // BLOCK], at % BLOCK
    # the block that a sequence's first new token lands in, and how many tokens it holds
    first, held = table[torch.arange(len(start), device=cu.device), start // BLOCK], start % BLOCK
    old = (torch.arange(BLOCK, device=cu.device)[None, :] < held[:, None])[:, None, :, None]
    new = dict(k=_rotated(s["k"].float(), *_angles(s, 1.0), s["case"]["interleaved"]), v=s["v"].float())
    for name in ("k", "v"):
        x = new[name].transpose(0, 1)                                         # [tokens, hkv, d]
        scale, codes = c[name + "_scale"], c[name]
        amax = torch.zeros_like(scale)
        amax.scatter_reduce_(0, block[:, None].expand(-1, x.shape[1]), x.abs().amax(-1), "amax")
        want = _power_scale(amax)
        before = scale[first]                                                 # [seqs, hkv]
        more = torch.where(amax[first] > 0, torch.maximum(before, want[first]), before)
        grown = torch.where((held > 0)[:, None], more, want[first])
        scale[block] = want[block]
        scale[first] = grown
        there = codes[first].view(torch.float8_e4m3fn).float() * (before / grown)[:, :, None, None]
        codes[first] = torch.where(old, _codes(there), codes[first])
        codes[block, :, slot] = _codes(x / scale[block][:, :, None])
    return _pools(c)


def _values(codes, scale, table):
    """[hkv, tokens, d] fp32 of the blocks of one sequence."""
    x = codes[table].view(torch.float8_e4m3fn).float() * scale[table][:, :, None, None]
    return x.transpose(0, 1).reshape(codes.shape[1], -1, codes.shape[3])


def _plain_chunk(s):
    c, q, case = s["cache"], s["q"], s["case"]
    hq, tokens, d = q.shape
    hkv = case["hkv"]
    o = torch.empty(tokens, hq, d, dtype=q.dtype, device=q.device).transpose(0, 1)
    lse = torch.empty(hq, tokens, dtype=torch.float32, device=q.device)
    at = 0
    for i, (n, p) in enumerate(zip(s["lens"], _past(case))):
        table = s["table"][i, : -(-(n + p) // BLOCK)].long()
        k, v = _values(c["k"], c["k_scale"], table)[:, : n + p], _values(c["v"], c["v_scale"], table)[:, : n + p]
        hidden = torch.ones(n, n + p, dtype=torch.bool, device=q.device).triu_(p + 1)
        for h in range(hkv):                                  # one KV head's scores at a time: they are large
            group, rows = slice(h * (hq // hkv), (h + 1) * (hq // hkv)), slice(at, at + n)
            x = torch.matmul(q[group, rows].float(), k[h].t()).mul_(d ** -0.5)
            x.masked_fill_(hidden, float("-inf"))
            top = x.amax(-1, keepdim=True)
            x = x.sub_(top).exp_()
            total = x.sum(-1, keepdim=True)
            o[group, rows] = (torch.matmul(x, v[h]) / total).to(q.dtype)
            lse[group, rows] = (top + total.log()).squeeze(-1)
        at += n
    return dict(o=o, lse=lse)


_PLAIN = dict(rope=_plain_rope, append=_plain_append, chunk=_plain_chunk)


# ------------------------------------------------------------------ 64 bits, from the definitions
def exact(case, seed):
    s = prepare(case, seed)
    return _EXACT[case["op"]](s, case)


def _turn(x, s, case, sign):
    """Each pair as a complex number times exp(i angle); x [..., t, d] float64."""
    freq, axis = _frequencies(case)
    y, n = x.clone(), len(freq)
    for i in range(n):
        a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + n)
        angle = s["positions"][axis[i]].double() * freq[i] * sign
        z = torch.complex(x[..., a], x[..., b]) * torch.polar(torch.ones_like(angle), angle)
        y[..., a], y[..., b] = z.real, z.imag
    return y


def _exact_rope(s, case):
    out = {}
    for name in ("q", "k"):
        y = _turn(s[name].double(), s, case, -1 if case["inverse"] else 1)
        out[name] = y.contiguous() if case["batched"] else y.transpose(0, 1).contiguous().transpose(0, 1)
    return out


def _decode(codes):
    """e4m3 codes to float64: sign, 4 exponent bits (bias 7), 3 mantissa bits."""
    c = codes.long()
    e, m = (c >> 3) & 15, (c & 7).double()
    mag = torch.where(e > 0, (1 + m / 8) * torch.exp2((e - 7).double()), m * 2.0 ** -9)
    return torch.where(c >= 128, -mag, mag)


def _round(x):
    """float64 to the nearest e4m3 value, ties to even: steps of 2^(exponent - 3), at least 2^-9."""
    step = torch.exp2((torch.frexp(x).exponent - 4).clamp_min(-9).double())
    return torch.round(x / step) * step


def _scale_of(x):
    """Smallest power of two s (as an exponent search) with max|x| / s <= 448, over the last two dimensions."""
    top = x.abs().amax((-1, -2))
    e = torch.ceil(torch.log2(torch.where(top > 0, top, 448.0) / 448.0))
    e = torch.where(top > 448.0 * torch.exp2(e), e + 1, e)                # log2 may be off by a rounding
    e = torch.where(top <= 448.0 * torch.exp2(e - 1), e - 1, e)
    return torch.where(top > 0, torch.exp2(e.clamp_min(-126)), 1.0)


def _exact_append(s, case):
    c, d, hkv = s["cache"], case["d"], case["hkv"]
    out = {}
    cu, past, table = s["cu"].tolist(), s["start"].tolist(), s["table"].tolist()
    new = dict(k=_turn(s["k"].double(), s, case, 1), v=s["v"].double())
    for name in ("k", "v"):
        codes, scale = _decode(c[name]), c[name + "_scale"].double()
        for b in range(case["seqs"]):
            n, p = cu[b + 1] - cu[b], past[b]
            b0, b1 = p // BLOCK, -(-(p + n) // BLOCK)
            ids = table[b][b0:b1]
            x = torch.zeros(hkv, (b1 - b0) * BLOCK, d, dtype=torch.float64, device="cuda")
            lo = p - b0 * BLOCK
            x[:, lo:lo + n] = new[name][:, cu[b]:cu[b + 1]]
            x = x.view(hkv, b1 - b0, BLOCK, d).transpose(0, 1)
            want = _scale_of(x)
            if lo:
                old = scale[ids[0]]
                want[0] = torch.where((x[0] != 0).any(-1).any(-1), torch.maximum(want[0], old), old)
            y = _round(x / want[:, :, None, None])
            z = codes[ids].clone()
            if lo:
                z[0, :, :lo] = _round(z[0, :, :lo] * (scale[ids[0]] / want[0])[:, None, None])
            at = torch.arange((b1 - b0) * BLOCK, device="cuda").view(-1, BLOCK)
            codes[ids] = torch.where(((at >= lo) & (at < lo + n))[:, None, :, None], y, z)
            scale[ids] = want
        out[name], out[name + "_scale"] = codes, scale
    return dict(k=out["k"], v=out["v"], k_scale=out["k_scale"], v_scale=out["v_scale"])


def _exact_chunk(s, case):
    if work(case)["flops"] > 4e12:
        return None
    c, hq, d = s["cache"], case["hq"], case["d"]
    o = torch.empty(sum(s["lens"]), hq, d, dtype=torch.float64, device="cuda")
    lse = torch.empty(hq, sum(s["lens"]), dtype=torch.float64, device="cuda")
    ends, held = s["cu"].tolist(), s["lengths"].tolist()
    for b, n in enumerate(held):
        a, e = ends[b], ends[b + 1]
        ids = s["table"][b, : -(-n // BLOCK)].long()
        for h in range(case["hkv"]):
            kd, vd = ((_decode(c[x][ids, h]) * c[x + "_scale"][ids, h].double()[:, None, None]).view(-1, d)[:n]
                      for x in ("k", "v"))
            for g in range(h * hq // case["hkv"], (h + 1) * hq // case["hkv"]):
                for i in range(a, e, 1024):                               # a slab of rows
                    j = min(e, i + 1024)
                    z = s["q"][g, i:j].double() @ kd.T / d ** 0.5
                    newest = torch.arange(i - a, j - a, device="cuda") + n - (e - a)
                    z = torch.where(torch.arange(n, device="cuda")[None, :] > newest[:, None], -torch.inf, z)
                    lse[g, i:j] = torch.logsumexp(z, 1)
                    o[i:j, g] = torch.exp(z - lse[g, i:j, None]) @ vd
    return dict(o=o.transpose(0, 1), lse=lse)


_EXACT = dict(rope=_exact_rope, append=_exact_append, chunk=_exact_chunk)
