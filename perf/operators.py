"""Measured cases of the serving operators: attention over packed prompts, the 8-bit cache's append, the attention over
that cache, and eviction from it.

`run` computes a case in elementary torch operations when `own` is false, and through the library's entry points when
it is true. `exact` computes the same outputs from the definitions in 64 bits.
"""
import random

import torch

own = False

BLOCK = 64          # tokens per cache block: one scale per block and KV head


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a few short requests: what one arriving user costs, latency counts
        dict(name="prompt_short", op="prompt", seqs=3, tokens=203, hq=8, hkv=2, d=64, token_major=True),
        # an ordinary batch of mixed prompts on a layer with eight query heads per KV head
        dict(name="prompt_mixed", op="prompt", seqs=24, tokens=16384, hq=64, hkv=8, d=128, token_major=True),
        # a long document among short ones, the largest
        dict(name="prompt_long", op="prompt", seqs=5, tokens=32768, hq=32, hkv=8, d=128, token_major=False),
        # one decoding step of a batch: one token appended to each sequence
        dict(name="append_step", op="append", seqs=64, tokens=64, past=2000, hkv=8, d=128, token_major=True),
        # prompts written to the cache, most of them behind tokens that are there
        dict(name="append_prompts", op="append", seqs=9, tokens=30011, past=500, hkv=8, d=128, token_major=True),
        # one user's next token after a short chat: latency
        dict(name="cache_one_short", op="cache", seqs=1, nq=1, longest=300, hq=32, hkv=8, d=128, weights=False),
        # an ordinary decoding batch of different lengths
        dict(name="cache_batch", op="cache", seqs=32, nq=1, longest=8192, hq=64, hkv=8, d=128, weights=False),
        # two users with long documents: few rows, the length has to be split
        dict(name="cache_long", op="cache", seqs=2, nq=1, longest=131072, hq=64, hkv=8, d=128, weights=False),
        # four drafted tokens checked at once, wide heads without groups
        dict(name="cache_draft_wide", op="cache", seqs=6, nq=4, longest=5000, hq=16, hkv=16, d=256, weights=False),
        # a step that also adds up the attention weights that eviction goes by
        dict(name="cache_weights", op="cache", seqs=16, nq=1, longest=16384, hq=32, hkv=8, d=128, weights=True),
        # a small cache cut to a quarter
        dict(name="evict_short", op="evict", seqs=2, longest=517, keep=130, recent=32, hkv=4, d=64),
        # long caches cut to an eighth
        dict(name="evict_long", op="evict", seqs=8, longest=32768, keep=4096, recent=512, hkv=8, d=128),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, evenly over the logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["prompt", "append", "cache", "cache", "evict"])
    if op == "prompt":
        hq, hkv = rng.choice([(8, 2), (16, 16), (32, 8), (12, 4), (6, 1)])
        tokens = _log(rng, 64, 16384)
        return dict(op=op, seqs=rng.randint(1, min(32, tokens)), tokens=tokens, hq=hq, hkv=hkv,
                    d=rng.choice([64, 128, 40, 80, 96, 112]), token_major=rng.random() < 0.5)
    if op == "append":
        seqs = _log(rng, 1, 96)
        tokens = seqs if rng.random() < 0.4 else _log(rng, seqs, 30000)
        return dict(op=op, seqs=seqs, tokens=tokens, past=_log(rng, 1, 1500), hkv=rng.choice([1, 2, 5, 8]),
                    d=rng.choice([64, 128, 256, 80, 112, 192]), token_major=rng.random() < 0.5)
    if op == "cache":
        hq, hkv = rng.choice([(32, 8), (64, 8), (16, 16), (8, 1), (12, 4), (20, 2), (7, 7)])
        seqs = _log(rng, 1, 64)
        return dict(op=op, seqs=seqs, nq=rng.choice([1, 1, 1, 2, 5]), longest=_log(rng, 1, min(60000, 400000 // seqs)),
                    hq=hq, hkv=hkv, d=rng.choice([64, 128, 128, 256, 80, 48, 192]), weights=rng.random() < 0.4)
    seqs, longest = _log(rng, 1, 8), _log(rng, 3, 20000)
    keep = rng.randint(1, max(1, longest // 2))
    return dict(op=op, seqs=seqs, longest=longest, keep=keep, recent=rng.randint(0, keep), hkv=rng.choice([1, 2, 5, 8]),
                d=rng.choice([64, 128, 256, 80]))


def _lengths(case):
    """The sequences' lengths: the case's own, whatever the seed. Prompts and appended tokens share out `tokens` (one
    each where there are as many as sequences); cached lengths lie between a quarter of the longest and the longest."""
    rng = random.Random("%s %s %s" % (case["op"], case["seqs"], case.get("tokens", case.get("longest"))))
    n = case["seqs"]
    if "tokens" in case:
        share = [rng.random() ** 2 + 0.02 for _ in range(n)]
        lens = [1 + int((case["tokens"] - n) * x / sum(share)) for x in share]
        lens[share.index(max(share))] += case["tokens"] - sum(lens)
        return lens
    lens = [rng.randint(max(1, case["longest"] // 4), case["longest"]) for _ in range(n)]
    lens[rng.randrange(n)] = case["longest"]
    return lens


def _past(case):
    """Tokens held before an append: none for the first sequence of several, up to `past` for the others."""
    rng = random.Random("past %s %s" % (case["seqs"], case["past"]))
    return [0 if i == 0 and case["seqs"] > 1 else rng.randint(1, case["past"]) for i in range(case["seqs"])]


def work(case):
    lens, d, hkv = _lengths(case), case["d"], case["hkv"]
    total = sum(lens)
    if case["op"] == "prompt":
        hq = case["hq"]
        return {"bytes": 2.0 * d * total * (2 * hq + 2 * hkv) + 4.0 * hq * total,
                "flops": 4.0 * hq * d * sum(n * (n + 1) / 2 for n in lens)}
    if case["op"] == "append":
        return {"bytes": 2.0 * total * hkv * d * (2 + 1), "flops": 0.0}
    if case["op"] == "cache":
        hq, nq = case["hq"], case["nq"]
        rows = case["seqs"] * hq * nq
        b = 2.0 * total * hkv * d + 4.0 * rows * d + 4.0 * rows + 8.0 * hkv * sum(-(-n // BLOCK) for n in lens)
        return {"bytes": b + (8.0 * total * hkv if case["weights"] else 0.0), "flops": 4.0 * hq * nq * d * total}
    kept = sum(min(n, case["keep"]) for n in lens)
    return {"bytes": 4.0 * total * hkv + kept * hkv * (4.0 * d + 8.0 + 4.0), "flops": 0.0}


# ------------------------------------------------------------------ inputs
def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def _heads(gen, heads, tokens, d, token_major):
    """[heads, tokens, d] bf16, as a projection leaves it ([tokens, heads, d] in memory) or head by head."""
    if token_major:
        return _randn(gen, tokens, heads, d).to(torch.bfloat16).transpose(0, 1)
    return _randn(gen, heads, tokens, d).to(torch.bfloat16)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _cumulative(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return _ints(at)


def _cache(gen, blocks, hkv, d):
    """A pool in use: codes of normal values (K and V of magnitude about 1), scales powers of two that differ by block
    and head, weights as some steps leave them."""
    codes = [(_randn(gen, blocks, hkv, BLOCK, d) * 48).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
             for _ in range(2)]
    scales = [torch.exp2(torch.randint(-7, -4, (blocks, hkv), generator=gen, device="cuda").float()) for _ in range(2)]
    weight = torch.rand(blocks, hkv, BLOCK, generator=gen, device="cuda").square_()
    return dict(k=codes[0], v=codes[1], k_scale=scales[0], v_scale=scales[1], weight=weight)


def _table(gen, lens, spare):
    """Block table over a pool of shuffled blocks, and the pool's size; `spare` more blocks for each sequence."""
    need = [-(-n // BLOCK) for n in lens]
    width = max(need) + spare
    blocks = len(lens) * width + 3
    perm = torch.randperm(blocks, generator=gen, device="cuda")[: len(lens) * width]
    return perm.to(torch.int32).view(len(lens), width).contiguous(), blocks


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    lens, d, hkv = _lengths(case), case["d"], case["hkv"]
    s = dict(case=case, lens=lens)
    if case["op"] == "prompt":
        for name, heads in (("q", case["hq"]), ("k", hkv), ("v", hkv)):
            s[name] = _heads(gen, heads, sum(lens), d, case["token_major"])
        s["cu"] = _cumulative(lens)
        return s
    if case["op"] == "append":
        past = _past(case)
        s["table"], blocks = _table(gen, [a + b for a, b in zip(past, lens)], 0)
        s["cache"] = _cache(gen, blocks, hkv, d)
        # a token now and then is larger than what its block holds, and the block's scale has to grow
        s["k"], s["v"] = (_heads(gen, hkv, sum(lens), d, case["token_major"]) * 4 for _ in range(2))
        s["cu"], s["start"] = _cumulative(lens), _ints(past)
        return s
    if case["op"] == "cache":
        s["table"], blocks = _table(gen, lens, 1)
        s["cache"] = _cache(gen, blocks, hkv, d)
        s["q"] = _randn(gen, case["seqs"], case["hq"], case["nq"], d).to(torch.bfloat16)
        s["lengths"] = _ints(lens)
        return s
    s["table"], blocks = _table(gen, lens, 0)
    room = -(-case["keep"] // BLOCK)
    s["cache"] = _cache(gen, blocks + case["seqs"] * room, hkv, d)
    s["to"] = (blocks + torch.randperm(case["seqs"] * room, generator=gen, device="cuda")).to(torch.int32)
    s["to"] = s["to"].view(case["seqs"], room).contiguous()
    s["lengths"] = _ints(lens)
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return _OWN[op](state)
    return _PLAIN[op](state)


def _pools(c, weight):
    """The cache as outputs: codes as the e4m3 values they are, and their scales."""
    out = dict(k=c["k"].view(torch.float8_e4m3fn), v=c["v"].view(torch.float8_e4m3fn), k_scale=c["k_scale"],
               v_scale=c["v_scale"])
    return dict(out, weight=c["weight"]) if weight else out


def _own_prompt(s):
    import exact_attention_79_gb300 as fa
    o, lse = fa.fwd_packed(s["q"], s["k"], s["v"], s["cu"], causal=True)
    return dict(o=o, lse=lse)


def _own_append(s):
    import exact_attention_79_gb300 as fa
    fa.cache8_append(fa.Cache8(**s["cache"]), s["k"], s["v"], s["cu"], s["table"], s["start"])
    return _pools(s["cache"], True)


def _own_cache(s):
    import exact_attention_79_gb300 as fa
    weights = s["case"]["weights"]
    o, lse = fa.fwd_cache8(s["q"], fa.Cache8(**s["cache"]), s["table"], s["lengths"], causal=True,
                           weight_decay=0.875 if weights else None)
    return dict(o=o, lse=lse, weight=s["cache"]["weight"]) if weights else dict(o=o, lse=lse)


def _own_evict(s):
    import exact_attention_79_gb300 as fa
    new, kept = fa.cache8_evict(fa.Cache8(**s["cache"]), s["table"], s["lengths"], s["case"]["keep"],
                                s["case"]["recent"], s["to"])
    return dict(_pools(s["cache"], True), lengths=new, kept=kept)


_OWN = dict(prompt=_own_prompt, append=_own_append, cache=_own_cache, evict=_own_evict)


# ---- plain forms
def _plain_prompt(s):
    q, k, v, d = s["q"], s["k"], s["v"], s["case"]["d"]
    hq, tokens = q.shape[0], q.shape[1]
    hkv = k.shape[0]
    o = torch.empty(tokens, hq, d, dtype=q.dtype, device=q.device).transpose(0, 1) if s["case"]["token_major"] else \
        torch.empty(hq, tokens, d, dtype=q.dtype, device=q.device)
    lse = torch.empty(hq, tokens, dtype=torch.float32, device=q.device)
    at = 0
    for n in s["lens"]:
        rows = slice(at, at + n)
        hidden = torch.ones(n, n, dtype=torch.bool, device=q.device).triu_(1)
        for h in range(hkv):                                  # one KV head's scores at a time: they are n x n each
            group = slice(h * (hq // hkv), (h + 1) * (hq // hkv))
            x = torch.matmul(q[group, rows].float(), k[h, rows].float().t()).mul_(d ** -0.5)
            x.masked_fill_(hidden, float("-inf"))
            top = x.amax(-1, keepdim=True)
            x = x.sub_(top).exp_()
            total = x.sum(-1, keepdim=True)
            o[group, rows] = (torch.matmul(x, v[h, rows].float()) / total).to(q.dtype)
            lse[group, rows] = (top + total.log()).squeeze(-1)
        at += n
    return dict(o=o, lse=lse)


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
    for name in ("k", "v"):
        x = s[name].transpose(0, 1).float()                                   # [tokens, hkv, d]
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
    c["weight"][block, :, slot] = 0
    return _pools(c, True)


def _values(codes, scale, table):
    """[B, hkv, width * 64, d] fp32 of the blocks of a table."""
    b, w = table.shape
    x = codes[table].view(torch.float8_e4m3fn).float() * scale[table][:, :, :, None, None]
    return x.permute(0, 2, 1, 3, 4).reshape(b, codes.shape[1], w * BLOCK, codes.shape[3])


def _plain_cache(s):
    c, q, table, case = s["cache"], s["q"], s["table"].long(), s["case"]
    b, hq, nq, d = q.shape
    hkv = case["hkv"]
    k, v = _values(c["k"], c["k_scale"], table), _values(c["v"], c["v_scale"], table)
    x = torch.matmul(q.float().view(b, hkv, -1, d), k.transpose(2, 3)).mul_(d ** -0.5).view(b, hq, nq, -1)
    key = torch.arange(x.shape[-1], device=q.device)
    last = s["lengths"].long()[:, None] - nq + torch.arange(nq, device=q.device)[None, :]    # newest visible key
    x = x.masked_fill_(key[None, None, None, :] > last[:, None, :, None], float("-inf"))
    top = x.amax(-1, keepdim=True)
    p = (x - top.clamp_min(torch.finfo(torch.float32).min)).exp_()
    total = p.sum(-1, keepdim=True)
    lse = (top + total.log()).squeeze(-1)
    some = torch.where(total > 0, total, torch.ones_like(total))
    v = torch.where(key[:, None] < s["lengths"][:, None, None, None], v, 0.0)
    o = torch.matmul(p.view(b, hkv, -1, p.shape[-1]), v)
    o = (o.view(b, hq, nq, d) / some).to(q.dtype)
    if not case["weights"]:
        return dict(o=o, lse=lse)
    add = (p / some).view(b, hkv, -1, p.shape[-1]).sum(2).view(b, hkv, -1, BLOCK).transpose(1, 2)
    held = (key < s["lengths"][:, None]).view(b, -1, 1, BLOCK)
    before = c["weight"][table]
    c["weight"][table] = torch.where(held, 0.875 * before + add, before)
    return dict(o=o, lse=lse, weight=c["weight"])


def _plain_evict(s):
    c, table, to, keep = s["cache"], s["table"].long(), s["to"].long(), s["case"]["keep"]
    b, w = table.shape
    hkv = c["k"].shape[1]
    n = s["lengths"].long()[:, None, None]
    score = c["weight"][table].transpose(1, 2).reshape(b, hkv, -1)
    at = torch.arange(score.shape[-1], device=score.device)
    score = torch.where(at >= n - s["case"]["recent"], float("inf"), score)   # the recent ones first
    score = torch.where(at < n, score, float("-inf"))
    order = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :keep]
    order = torch.where(order < n, order, w * BLOCK).sort(-1).values          # in their order, absent ones last
    fill = to.shape[1] * BLOCK - order.shape[-1]
    src = torch.cat([order, order.new_full((b, hkv, fill), w * BLOCK)], -1)
    there = (src < w * BLOCK).view(b, hkv, -1, BLOCK)
    src = src.clamp_max(w * BLOCK - 1)
    blk = torch.gather(table[:, None].expand(b, hkv, w), 2, src // BLOCK)
    head = torch.arange(hkv, device=n.device)[None, :, None]
    dst = to[:, None].expand(b, hkv, -1)                                      # [b, hkv, room]
    heads = head.expand_as(dst)
    used = there.any(-1)
    for name in ("k", "v"):
        scale = c[name + "_scale"]
        x = c[name][blk, head, src % BLOCK].view(torch.float8_e4m3fn).float() * scale[blk, head][..., None]
        x = x.view(b, hkv, -1, BLOCK, x.shape[-1])
        want = _power_scale(torch.where(there[..., None], x.abs(), 0.0).amax((-1, -2)))
        scale[dst, heads] = torch.where(used, want, scale[dst, heads])
        c[name][dst, heads] = torch.where(there[..., None], _codes(x / want[..., None, None]), c[name][dst, heads])
    moved = c["weight"][blk, head, src % BLOCK].view(b, hkv, -1, BLOCK)
    c["weight"][dst, heads] = torch.where(there, moved, c["weight"][dst, heads])
    kept = torch.where(order < w * BLOCK, order, -1).to(torch.int32)
    if kept.shape[-1] < keep:
        kept = torch.cat([kept, kept.new_full((b, hkv, keep - kept.shape[-1]), -1)], -1)
    return dict(_pools(c, True), lengths=s["lengths"].clamp_max(keep), kept=kept)


_PLAIN = dict(prompt=_plain_prompt, append=_plain_append, cache=_plain_cache, evict=_plain_evict)


# ------------------------------------------------------------------ 64 bits, from the definitions
def exact(case, seed):
    s = prepare(case, seed)
    return _EXACT[case["op"]](s, case)


def _exact_prompt(s, case):
    if work(case)["flops"] > 8e12:
        return None
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    o = torch.empty(hq, sum(s["lens"]), d, dtype=torch.float64, device="cuda")
    lse = torch.empty(hq, sum(s["lens"]), dtype=torch.float64, device="cuda")
    ends = s["cu"].tolist()
    for h in range(hq):
        for a, b in zip(ends[:-1], ends[1:]):
            kd, vd = (s[x][h * hkv // hq, a:b].double() for x in ("k", "v"))
            for i in range(a, b, 2048):                                   # a slab of rows sees the keys up to its end
                j = min(b, i + 2048)
                z = s["q"][h, i:j].double() @ kd[: j - a].T / d ** 0.5
                late = torch.arange(j - a, device="cuda")[None, :] > torch.arange(i - a, j - a, device="cuda")[:, None]
                z = torch.where(late, -torch.inf, z)
                lse[h, i:j] = torch.logsumexp(z, 1)
                o[h, i:j] = torch.exp(z - lse[h, i:j, None]) @ vd[: j - a]
    if case["token_major"]:
        o = o.transpose(0, 1).contiguous().transpose(0, 1)
    return dict(o=o, lse=lse)


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
    for name in ("k", "v"):
        codes, scale = _decode(c[name]), c[name + "_scale"].double()
        for b in range(case["seqs"]):
            n, p = cu[b + 1] - cu[b], past[b]
            b0, b1 = p // BLOCK, -(-(p + n) // BLOCK)
            ids = table[b][b0:b1]
            x = torch.zeros(hkv, (b1 - b0) * BLOCK, d, dtype=torch.float64, device="cuda")
            lo = p - b0 * BLOCK
            x[:, lo:lo + n] = s[name][:, cu[b]:cu[b + 1]].double()
            x = x.view(hkv, b1 - b0, BLOCK, d).transpose(0, 1)
            want = _scale_of(x)
            if lo:
                old = scale[ids[0]]
                want[0] = torch.where((x[0] != 0).any((-1, -2)), torch.maximum(want[0], old), old)
            y = _round(x / want[:, :, None, None])
            z = codes[ids].clone()
            if lo:
                z[0, :, :lo] = _round(z[0, :, :lo] * (scale[ids[0]] / want[0])[:, None, None])
            at = torch.arange((b1 - b0) * BLOCK, device="cuda").view(-1, BLOCK)
            codes[ids] = torch.where(((at >= lo) & (at < lo + n))[:, None, :, None], y, z)
            scale[ids] = want
        out[name], out[name + "_scale"] = codes, scale
    w = c["weight"].double()
    for b in range(case["seqs"]):
        at = torch.arange(past[b], past[b] + cu[b + 1] - cu[b], device="cuda")
        w[s["table"][b].long()[at // BLOCK], :, at % BLOCK] = 0
    return dict(out, weight=w)


def _exact_cache(s, case):
    c, q = s["cache"], s["q"].double()
    b, hq, nq, d = q.shape
    g = hq // case["hkv"]
    o, lse = torch.zeros_like(q), torch.full((b, hq, nq), -torch.inf, dtype=torch.float64, device="cuda")
    w = c["weight"].double()
    for i, n in enumerate(s["lens"]):
        ids = s["table"][i, : -(-n // BLOCK)].long()
        for h in range(case["hkv"]):
            kd, vd = ((_decode(c[x][ids, h]) * c[x + "_scale"][ids, h].double()[:, None, None]).view(-1, d)[:n]
                      for x in ("k", "v"))
            total = torch.zeros(n, dtype=torch.float64, device="cuda")
            for r in range(nq):
                m = n - nq + r + 1                                            # keys that query r sees
                if m <= 0:
                    continue
                z = q[i, h * g:(h + 1) * g, r] @ kd[:m].T * d ** -0.5
                lse[i, h * g:(h + 1) * g, r] = torch.logsumexp(z, 1)
                p = torch.softmax(z, 1)
                o[i, h * g:(h + 1) * g, r] = p @ vd[:m]
                total[:m] += p.sum(0)
            row = torch.arange(n, device="cuda")
            w[ids[row // BLOCK], h, row % BLOCK] = 0.875 * w[ids[row // BLOCK], h, row % BLOCK] + total
    return dict(o=o, lse=lse, weight=w) if case["weights"] else dict(o=o, lse=lse)


def _exact_evict(s, case):
    c = s["cache"]
    out = {x: _decode(c[x]) for x in ("k", "v")}
    out.update({x: c[x].double() for x in ("k_scale", "v_scale", "weight")})
    kept = torch.full((case["seqs"], case["hkv"], case["keep"]), -1, dtype=torch.int32, device="cuda")
    new = [min(n, case["keep"]) for n in s["lens"]]
    for i, n in enumerate(s["lens"]):
        ids, to = s["table"][i].long(), s["to"][i].long()
        for h in range(case["hkv"]):
            row = torch.arange(n, device="cuda")
            w = c["weight"][ids[row // BLOCK], h, row % BLOCK].double()
            old = max(0, n - case["recent"])
            pick = torch.argsort(-w[:old], stable=True)[: new[i] - (n - old)] if n > case["keep"] else row[:old]
            pick = torch.cat([pick, row[old:]]).sort().values
            kept[i, h, : len(pick)] = pick.int()
            for blk in range(0, len(pick), BLOCK):
                part, t = pick[blk:blk + BLOCK], to[blk // BLOCK]
                at = (ids[part // BLOCK], h, part % BLOCK)
                for x in ("k", "v"):
                    y = _decode(c[x][at]) * c[x + "_scale"][at[0], h].double()[:, None]
                    scale = _scale_of(y)
                    out[x][t, h, : len(part)] = _round(y / scale)
                    out[x + "_scale"][t, h] = scale
                out["weight"][t, h, : len(part)] = w[part]
    return dict(out, lengths=_ints(new), kept=kept)


_EXACT = dict(prompt=_exact_prompt, append=_exact_append, cache=_exact_cache, evict=_exact_evict)
