"""Cases of the attention-layer operators of the library, with their plain forms.

Four operators that a serving step of an attention layer runs one after another:

* ``qk_norm_rope``: RMS norm of every query and key head, and the position rotation;
* ``kv_append``: new K / V rows into a paged 8-bit cache with one scale per (block of
  tokens, head);
* ``attention``: queries against that cache, for prompts and for single tokens;
* ``matvec``: projections of a few tokens with 4-bit weights and group scales.

``run`` computes an operator in elementary torch operations, or, with ``own`` set, by
the library's own call.  ``exact`` states the same operator in 64 bits.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0
MIN_EXP = -100  # smallest exponent of a cache block's power-of-two scale
EPS = 1e-6


# ------------------------------------------------------------------------- cases
def listed():
    attn = dict(op="attention", heads=48, kv_heads=8, head_dim=128, block=64, causal=True, ragged=False)
    return [
        # one user's next token after a short prompt: the smallest call, latency alone
        dict(attn, name="attn_token_1x700", n_seqs=1, q_len=1, kv_len=700),
        # next tokens of 32 users whose texts have different lengths
        dict(attn, name="attn_token_32x8192", n_seqs=32, q_len=1, kv_len=8192, ragged=True),
        # next tokens of two long documents, wide heads, small cache blocks
        dict(attn, name="attn_token_2x131072", n_seqs=2, q_len=1, kv_len=131072, heads=24, kv_heads=4,
             head_dim=256, block=16, ragged=True),
        # four prompts of odd lengths in one batch
        dict(attn, name="attn_prompt_4x3001", n_seqs=4, q_len=3001, kv_len=3001, ragged=True),
        # one long prompt
        dict(attn, name="attn_prompt_8192", n_seqs=1, q_len=8192, kv_len=8192),
        # a slice of a long prompt against what the cache holds of it, wide heads
        dict(attn, name="attn_slice_1024_of_32768", n_seqs=1, q_len=1024, kv_len=32768, heads=24, kv_heads=4,
             head_dim=256),
        # the new token of 32 users
        dict(name="norm_rope_32", op="qk_norm_rope", tokens=32, heads=48, kv_heads=8, head_dim=128, rot_dim=128,
             interleaved=False),
        # a batch of prompts, rotation of a part of each head
        dict(name="norm_rope_32768", op="qk_norm_rope", tokens=32768, heads=48, kv_heads=8, head_dim=128, rot_dim=64,
             interleaved=False),
        # the new token of 32 users, into blocks that hold earlier tokens
        dict(name="append_32x1", op="kv_append", n_seqs=32, q_len=1, kv_len=1000, kv_heads=8, head_dim=128, block=64),
        # eight prompts that begin inside a block
        dict(name="append_8x4096", op="kv_append", n_seqs=8, q_len=4096, kv_len=4133, kv_heads=8, head_dim=128,
             block=64),
        # output projection of one token
        dict(name="matvec_1x5120x6144", op="matvec", tokens=1, n=5120, k=6144),
        # the MLP's fused gate and up projection of four tokens
        dict(name="matvec_4x34816x5120", op="matvec", tokens=4, n=34816, k=5120),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention"] * 5 + ["qk_norm_rope", "kv_append", "matvec"])
    d = rng.choice([64, 128, 128, 256])
    kvh = rng.choice([1, 2, 4, 8])
    if op == "qk_norm_rope":
        h = kvh * rng.choice([1, 2, 4, 6])
        return dict(op=op, tokens=_log(rng, 1, 20000), heads=h, kv_heads=kvh, head_dim=d,
                    rot_dim=rng.choice([16, 32, d // 2, d]), interleaved=rng.random() < 0.3)
    block = rng.choice([16, 32, 64, 128])
    if op == "kv_append":
        n = _log(rng, 1, 64)
        q = _log(rng, 1, 20000 // n)
        return dict(op=op, n_seqs=n, q_len=q, kv_len=q + rng.randrange(0, 500), kv_heads=kvh, head_dim=d, block=block)
    if op == "matvec":
        return dict(op=op, tokens=rng.randint(1, 16), n=16 * _log(rng, 16, 1100), k=64 * _log(rng, 4, 200))
    heads = kvh * rng.choice([1, 2, 3, 6, 8])
    case = dict(op=op, heads=heads, kv_heads=kvh, head_dim=d, block=block, causal=rng.random() < 0.85,
                ragged=rng.random() < 0.7)
    if rng.random() < 0.5:  # next tokens, or a few tokens to be verified
        n = _log(rng, 1, 64)
        q = rng.choice([1, 1, 1, 2, 3, 5])
        return dict(case, n_seqs=n, q_len=q, kv_len=q + _log(rng, 1, min(131072, 200_000_000 // (n * kvh * d))))
    n = rng.randint(1, 4)
    q = _log(rng, 9, min(4096, int(math.sqrt(2.5e9 / (n * heads)))))
    past = rng.choice([0, _log(rng, 1, 8192)])
    return dict(case, n_seqs=n, q_len=q, kv_len=q + min(past, int(2.5e9 / (n * heads * q))))


def _lengths(case):
    """(new tokens, total tokens) of each sequence: a ragged batch has lengths between an
    eighth and the whole of the case's."""
    n, q, kv = case["n_seqs"], case["q_len"], case["kv_len"]
    if not case.get("ragged"):
        return [q] * n, [kv] * n
    rng = random.Random(1000003 * n + 1009 * q + kv)
    q_lens, kv_lens = [], []
    for i in range(n):
        f = 1.0 if i == 0 else rng.uniform(0.125, 1.0)
        past = int((kv - q) * f)
        new = max(1, int(q * (1.0 if i == 0 else rng.uniform(0.125, 1.0)))) if q > 8 else q
        q_lens.append(new)
        kv_lens.append(past + new)
    return q_lens, kv_lens


def work(case):
    op = case["op"]
    if op == "qk_norm_rope":
        t, d, r = case["tokens"], case["head_dim"], case["rot_dim"]
        e = t * (case["heads"] + case["kv_heads"]) * d
        return {"bytes": 4 * e + t * (8 + 4 * r), "flops": 8 * e}
    if op == "matvec":
        t, n, k = case["tokens"], case["n"], case["k"]
        return {"bytes": n * k * 9 // 16 + 2 * t * (n + k), "flops": 2 * t * n * k}
    q_lens, kv_lens = _lengths(case)
    w = case["kv_heads"] * case["head_dim"]
    if op == "kv_append":
        new = sum(q_lens)
        # what a block holds of earlier tokens is rewritten only when its scale grows
        return {"bytes": new * w * 2 * 3, "flops": new * w * 2 * 3}
    h, d = case["heads"], case["head_dim"]
    pairs = 0
    for q, kv in zip(q_lens, kv_lens):
        pairs += q * kv - (q * (q - 1) // 2 if case["causal"] else 0)
    return {"bytes": 2 * sum(kv_lens) * w + 4 * sum(q_lens) * h * d, "flops": 4 * pairs * h * d}


# ------------------------------------------------------------------------ inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _block_scale(amax):
    """Smallest power of two s with 448 s >= amax (at least 2^MIN_EXP)."""
    m, e = torch.frexp(amax)  # amax = m 2^e, 0.5 <= m < 1; 448 = 0.875 * 2^9
    e = torch.where(m > 0.875, e - 8, e - 9)
    e = torch.where(amax > 0, e, torch.full_like(e, MIN_EXP)).clamp(min=MIN_EXP)
    return torch.ldexp(torch.ones_like(amax), e)


def _to_codes(x):
    return x.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)


def _filled_cache(case, kv_lens, g, rest_mask=0xFF):
    """A paged cache that holds kv_lens[s] tokens of every sequence: (k codes, v codes,
    k scales, v scales, block table with room for the case's longest).  Blocks are
    shuffled; places that no token holds have arbitrary bytes within rest_mask."""
    hk, d, b = case["kv_heads"], case["head_dim"], case["block"]
    n = len(kv_lens)
    per = -(-case["kv_len"] // b)
    lens = torch.tensor(kv_lens, device="cuda")
    count = n * per + 3
    table = torch.randperm(count, generator=g, device="cuda")[: n * per].reshape(n, per)
    held = torch.arange(per * b, device="cuda") < lens[:, None]
    codes, scales = [], []
    for spread in (0.2, 0.5):  # keys, values: how much the size of a token's row varies
        x = torch.randn((n, per * b, hk, d), generator=g, device="cuda")
        x *= torch.exp(spread * torch.randn((n, per * b, hk, 1), generator=g, device="cuda"))
        x = (x * held[:, :, None, None]).to(torch.bfloat16).float()
        x = x.reshape(n, per, b, hk, d).transpose(2, 3)
        s = _block_scale(x.abs().amax(dim=(3, 4)))
        c = _to_codes(x / s[..., None, None])
        rest = torch.randint(0, 256, c.shape, generator=g, device="cuda", dtype=torch.uint8)
        c = torch.where(held.reshape(n, per, 1, b, 1), c, rest & rest_mask)
        whole = torch.empty((count, hk, b, d), dtype=torch.uint8, device="cuda").fill_(0x7F & rest_mask)
        whole[table.reshape(-1)] = c.reshape(n * per, hk, b, d)
        sc = torch.ones((count, hk), device="cuda")
        sc[table.reshape(-1)] = s.reshape(n * per, hk)
        codes.append(whole)
        scales.append(sc)
    return codes[0], codes[1], scales[0], scales[1], table.to(torch.int32).contiguous()


def _sequences(q_lens, kv_lens):
    cu = torch.tensor([0] + q_lens).cumsum(0).to(device="cuda", dtype=torch.int32)
    return cu, torch.tensor(kv_lens, dtype=torch.int32, device="cuda")


def _e2m1_values():
    v = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device="cuda")
    return torch.cat([v, -v])


def _weight(n, k, g):
    """A 4-bit weight: codes [n, k/2] (even columns in the low nibble), E4M3 scales of 16
    columns in atoms of 128 rows x 4 groups (row r, group j at byte (r%32)*16 + (r/32)*4 + j),
    and the global scale that the products are divided by."""
    w = torch.randn((n, k), generator=g, device="cuda") * 0.02
    gs = 2688.0 / w.abs().amax()
    w = w.reshape(n, k // 16, 16)
    sf = (w.abs().amax(dim=2) / 6.0 * gs).to(torch.float8_e4m3fn)
    x = w * (gs / sf.float().clamp(min=2.0 ** -9))[..., None]
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    c = torch.bucketize(x.abs(), edges).to(torch.uint8) + 8 * (x < 0).to(torch.uint8)
    c = c.reshape(n, k // 2, 2)
    codes = (c[..., 0] | (c[..., 1] << 4)).contiguous()
    rows = -(-n // 128) * 128
    s = torch.zeros((rows, k // 16), dtype=torch.uint8, device="cuda")
    s[:n] = sf.view(torch.uint8)
    s = s.reshape(rows // 128, 4, 32, k // 64, 4).permute(0, 3, 2, 1, 4).contiguous().reshape(-1)
    return codes, s, gs.reshape(1).float()


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]
    state = {"case": case}
    if op == "matvec":
        x = torch.randn((case["tokens"], case["k"]), generator=g, device="cuda")
        codes, scales, gs = _weight(case["n"], case["k"], g)
        return dict(state, x=x.to(torch.bfloat16), codes=codes, scales=scales, gs=gs)
    hk, d = case["kv_heads"], case["head_dim"]
    if op == "qk_norm_rope":
        t, h, r = case["tokens"], case["heads"], case["rot_dim"]
        # q and k are column ranges of one fused projection's output, v behind them
        qkv = torch.randn((t, (h + 2 * hk) * d), generator=g, device="cuda")
        qkv = (qkv * torch.exp(torch.randn((t, 1), generator=g, device="cuda"))).to(torch.bfloat16)
        most = 40960
        angle = torch.arange(most, device="cuda", dtype=torch.float64)[:, None] * torch.pow(
            torch.tensor(10000.0, device="cuda", dtype=torch.float64),
            -torch.arange(0, r, 2, device="cuda", dtype=torch.float64) / r)
        table = torch.cat([angle.cos(), angle.sin()], dim=1).float()
        weights = (1.0 + 0.2 * torch.randn((2, d), generator=g, device="cuda")).to(torch.bfloat16)
        return dict(state, q=qkv[:, : h * d], k=qkv[:, h * d: (h + hk) * d], w_q=weights[0], w_k=weights[1],
                    positions=torch.randint(0, most, (t,), generator=g, device="cuda"), table=table)
    q_lens, kv_lens = _lengths(case)
    cu, lens = _sequences(q_lens, kv_lens)
    t = sum(q_lens)
    if op == "kv_append":
        # the cache holds the earlier tokens; the new rows are column ranges of wider rows
        past = [b - a for a, b in zip(q_lens, kv_lens)]
        kc, vc, ks, vs, table = _filled_cache(case, past, g, rest_mask=0x77)
        rows = torch.randn((t, 2 * hk * d), generator=g, device="cuda")
        rows = (rows * torch.exp(torch.randn((t, 1), generator=g, device="cuda"))).to(torch.bfloat16)
        return dict(state, k=rows[:, : hk * d], v=rows[:, hk * d:], cu=cu, lens=lens, table=table, cache=(kc, vc, ks, vs))
    kc, vc, ks, vs, table = _filled_cache(case, kv_lens, g)
    behind = torch.arange(table.shape[1], device="cuda") * case["block"] >= lens[:, None]
    table.masked_fill_(behind, -1)  # no block where a sequence has ended
    q = (1.5 * torch.randn((t, case["heads"] * d), generator=g, device="cuda")).to(torch.bfloat16)
    return dict(state, q=q, cu=cu, lens=lens, table=table, cache=(kc, vc, ks, vs), max_q=max(q_lens))


# ------------------------------------------------------------------- plain forms
def _plain_norm_rope(s):
    case = s["case"]
    d, r = case["head_dim"], case["rot_dim"]
    cs = s["table"][s["positions"]][:, None, :]
    cos, sin = cs[..., : r // 2], cs[..., r // 2:]

    def heads(x, w):
        x = x.float().reshape(x.shape[0], -1, d)
        x = x * torch.rsqrt((x * x).mean(dim=2, keepdim=True) + EPS) * w.float()
        a, b = (x[..., 0:r:2], x[..., 1:r:2]) if case["interleaved"] else (x[..., : r // 2], x[..., r // 2: r])
        y = (a * cos - b * sin, b * cos + a * sin)
        y = torch.stack(y, dim=3).flatten(2) if case["interleaved"] else torch.cat(y, dim=2)
        return torch.cat([y, x[..., r:]], dim=2).to(torch.bfloat16).flatten(1)

    return {"q": heads(s["q"], s["w_q"]), "k": heads(s["k"], s["w_k"])}


def _plain_append(s):
    case, (kc, vc, ks, vs) = s["case"], s["cache"]
    b = case["block"]
    cu, lens = s["cu"].long(), s["lens"].long()
    t = torch.arange(s["k"].shape[0], device="cuda")
    seq = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    past = lens[seq] - (cu[seq + 1] - cu[seq])
    pos = past + t - cu[seq]
    block = s["table"].long()[seq, pos // b]
    # how many earlier tokens each block that gets new ones holds, -1 for other blocks
    held = torch.full((kc.shape[0],), -1, device="cuda")
    held[block] = (past - pos // b * b).clamp(0, b)
    keep = (torch.arange(b, device="cuda") < held[:, None])[:, None, :, None]

    def write(rows, codes, scales):
        x = rows.float().reshape(t.numel(), case["kv_heads"], case["head_dim"])
        amax = torch.zeros_like(scales).index_reduce_(0, block, x.abs().amax(dim=2), "amax")
        new = _block_scale(amax)
        new = torch.where((held > 0)[:, None], torch.maximum(scales, new), new)
        new = torch.where((held >= 0)[:, None], new, scales)
        old = codes.view(torch.float8_e4m3fn).float() * (scales / new)[..., None, None]
        codes.copy_(torch.where(keep, _to_codes(old), codes))
        codes.transpose(1, 2)[block, pos % b] = _to_codes(x / new[block][..., None])
        scales.copy_(new)

    write(s["k"], kc, ks)
    write(s["v"], vc, vs)
    return _cache_values(s)


def _cache_values(s):
    kc, vc, ks, vs = s["cache"]
    return {"k": kc.view(torch.float8_e4m3fn), "v": vc.view(torch.float8_e4m3fn), "k_scales": ks, "v_scales": vs}


def _plain_attention(s):
    case, (kc, vc, ks, vs) = s["case"], s["cache"]
    hk, d, h = case["kv_heads"], case["head_dim"], case["heads"]
    cu, lens, table = s["cu"].long(), s["lens"].long(), s["table"].long().clamp(min=0)
    n, mq, mk = lens.numel(), s["max_q"], table.shape[1] * case["block"]
    q_lens = cu[1:] - cu[:-1]
    i, j = torch.arange(mq, device="cuda"), torch.arange(mk, device="cuda")
    held = j < lens[:, None]

    def gather(codes, scales):
        x = codes[table].view(torch.float8_e4m3fn).float() * scales[table][..., None, None]
        x = x.transpose(1, 2).reshape(n, hk, mk, d)
        return torch.where(held[:, None, :, None], x, 0.0)

    rows = (cu[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"].float()[rows].reshape(n, mq, hk, h // hk, d).permute(0, 2, 3, 1, 4)
    p = torch.matmul(q.reshape(n, hk, -1, d), gather(kc, ks).transpose(2, 3)).reshape(n, hk, h // hk, mq, mk)
    p *= d ** -0.5
    seen = held[:, None, :]
    if case["causal"]:
        seen = seen & (j <= (lens - q_lens)[:, None, None] + i[:, None])
    p.masked_fill_(~seen[:, None, None], -math.inf)
    most = p.amax(dim=4, keepdim=True)
    p.sub_(torch.where(most == -math.inf, 0.0, most)).exp_()
    total = p.sum(dim=4, keepdim=True)
    o = torch.matmul(p.reshape(n, hk, -1, mk), gather(vc, vs)).reshape(n, hk, h // hk, mq, d)
    o = o / torch.where(total == 0, 1.0, total)
    t = torch.arange(s["q"].shape[0], device="cuda")
    seq = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    return o.permute(0, 3, 1, 2, 4)[seq, t - cu[seq]].reshape(t.numel(), h * d).to(torch.bfloat16)


def _plain_matvec(s):
    n, k = s["case"]["n"], s["case"]["k"]
    c = torch.stack([s["codes"] & 15, s["codes"] >> 4], dim=2).long()
    w = _e2m1_values()[c].reshape(n, k // 16, 16)
    sf = s["scales"].view(torch.float8_e4m3fn).float().reshape(-1, k // 64, 32, 4, 4)
    sf = sf.permute(0, 3, 2, 1, 4).reshape(-1, k // 16)[:n]
    y = torch.matmul(s["x"].float(), (w * sf[..., None]).reshape(n, k).t())
    return (y / s["gs"]).to(torch.bfloat16)


# ------------------------------------------------------------------ library calls
def _own(s):
    import nvfp4_w4a4_quantized_02_b200 as nv
    case, op = s["case"], s["case"]["op"]
    if op == "matvec":
        w = nv.NVFP4Tensor(s["codes"], s["scales"], s["gs"], case["n"], case["k"])
        return nv.matvec(s["x"], w)
    if op == "qk_norm_rope":
        q, k = nv.qk_norm_rope(s["q"], s["k"], s["w_q"], s["w_k"], s["positions"], s["table"], eps=EPS,
                               interleaved=case["interleaved"])
        return {"q": q, "k": k}
    cache = nv.BlockKVCache(*s["cache"])
    if op == "kv_append":
        nv.kv_append(s["k"], s["v"], s["cu"], s["lens"], s["table"], cache)
        return _cache_values(s)
    return nv.attention(s["q"], s["cu"], s["lens"], s["table"], cache, causal=case["causal"])


def run(state):
    if own:
        return _own(state)
    return {"qk_norm_rope": _plain_norm_rope, "kv_append": _plain_append, "attention": _plain_attention,
            "matvec": _plain_matvec}[state["case"]["op"]](state)


# --------------------------------------------------------------- 64-bit statements
def _exact_rotation(s):
    case = s["case"]
    d, half = case["head_dim"], case["rot_dim"] // 2
    cs = s["table"].double()[s["positions"]]
    turn = torch.complex(cs[:, :half], cs[:, half:])[:, None, :]
    out = {}
    for name, w in (("q", s["w_q"]), ("k", s["w_k"])):
        x = s[name].double().unflatten(1, (-1, d))
        x = x / (x.square().sum(dim=2, keepdim=True) / d + EPS).sqrt() * w.double()
        z = x[..., : 2 * half]
        z = z.unflatten(2, (half, 2)) if case["interleaved"] else z.unflatten(2, (2, half)).transpose(2, 3)
        z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * turn)
        z = z.flatten(2) if case["interleaved"] else z.transpose(2, 3).flatten(2)
        out[name] = torch.cat([z, x[..., 2 * half:]], dim=2).flatten(1)
    return out


def _nearest_e4m3(x):
    """x rounded to the E4M3 grid, ties to even, magnitudes above 448 to 448."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(e - 3)
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def _exact_append(s):
    case = s["case"]
    b, hk, d = case["block"], case["kv_heads"], case["head_dim"]
    q_lens, kv_lens = _lengths(case)
    cu = s["cu"].tolist()
    table = s["table"].tolist()
    out = {}
    for name, codes, scales in (("k", s["cache"][0], s["cache"][2]), ("v", s["cache"][1], s["cache"][3])):
        values, sc = codes.view(torch.float8_e4m3fn).double(), scales.double().clone()
        rows = s[name].double().reshape(-1, hk, d)
        for i, (new, total) in enumerate(zip(q_lens, kv_lens)):
            past = total - new
            for n in range(past // b, -(-total // b)):
                at, first = table[i][n], max(past, n * b)
                x = rows[cu[i] + first - past: cu[i] + min(total, n * b + b) - past].transpose(0, 1)
                top = x.abs().amax(dim=(1, 2))
                scale = torch.exp2(torch.ceil(torch.log2((top / 448).clamp(min=2.0 ** MIN_EXP))))
                scale = torch.where(448 * scale / 2 >= top, scale / 2, scale).clamp(min=2.0 ** MIN_EXP)
                if first > n * b:
                    scale = torch.maximum(scale, sc[at])
                    old = values[at, :, : first - n * b]
                    values[at, :, : first - n * b] = _nearest_e4m3(old * (sc[at] / scale)[:, None, None])
                sc[at] = scale
                values[at, :, first - n * b: first - n * b + x.shape[1]] = _nearest_e4m3(x / scale[:, None, None])
        out[name], out[name + "_scales"] = values, sc
    return out


def _exact_attention(s):
    case, (kc, vc, ks, vs) = s["case"], s["cache"]
    hk, d, g = case["kv_heads"], case["head_dim"], case["heads"] // case["kv_heads"]
    q_lens, kv_lens = _lengths(case)
    out = torch.zeros((sum(q_lens), hk, g, d), dtype=torch.float64, device="cuda")
    q = s["q"].double().reshape(-1, hk, g, d)
    at = 0
    for i, (new, total) in enumerate(zip(q_lens, kv_lens)):
        blocks = s["table"][i, : -(-total // case["block"])].long()
        for a in range(hk):
            k = kc[blocks, a].view(torch.float8_e4m3fn).double() * ks[blocks, a].double()[:, None, None]
            v = vc[blocks, a].view(torch.float8_e4m3fn).double() * vs[blocks, a].double()[:, None, None]
            k, v = k.flatten(0, 1)[:total], v.flatten(0, 1)[:total]
            for first in range(0, new, 2048):
                rows = q[at + first: at + min(new, first + 2048), a]
                z = torch.einsum("igd,jd->gij", rows, k) / math.sqrt(d)
                if case["causal"]:
                    last = total - new + first + torch.arange(rows.shape[0], device="cuda")
                    z = z.masked_fill(torch.arange(total, device="cuda") > last[:, None], -math.inf)
                out[at + first: at + first + rows.shape[0], a] = torch.einsum("gij,jd->igd", torch.softmax(z, dim=2), v)
        at += new
    return out.flatten(1)


def _exact_matvec(s):
    n, k = s["case"]["n"], s["case"]["k"]
    x, out = s["x"].double(), []
    r = torch.arange(n, device="cuda")
    group = torch.arange(k // 16, device="cuda")
    at = ((r[:, None] // 128) * (k // 64) + group // 4) * 512 + (r[:, None] % 32) * 16 + (r[:, None] % 128) // 32 * 4 + group % 4
    sf = s["scales"][at].view(torch.float8_e4m3fn).double()
    for first in range(0, n, 4096):
        c = s["codes"][first: first + 4096].long()
        c = torch.stack([c % 16, c // 16], dim=2).flatten(1)
        e, m = c % 8 // 2, c % 2
        w = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * torch.exp2(e.double() - 1)) * (1 - 2 * (c // 8))
        w = w.unflatten(1, (-1, 16)) * sf[first: first + 4096, :, None]
        out.append(x @ w.flatten(1).t())
    return torch.cat(out, dim=1) / s["gs"].double()


def exact(case, seed):
    s = prepare(case, seed)
    return {"qk_norm_rope": _exact_rotation, "kv_append": _exact_append, "attention": _exact_attention,
            "matvec": _exact_matvec}[case["op"]](s)
