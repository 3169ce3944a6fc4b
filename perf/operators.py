"""The attention operators of a serving step, as they are measured: the append of rotated keys and
values to a paged 4-bit cache, and attention over that cache.

``run`` computes them in their plain form (elementary torch operations in fp32) or, with ``own``
set, through the library's entry points. ``exact`` is the definition in fp64.

Cache layout (uint8): ``[page][kv head][page_size / 16][16 (D + 8)]``. A block of 16 tokens holds
its K codes ``[16][D / 2]``, V codes ``[16][D / 2]``, K parameters ``[16][2]`` and V parameters
``[16][2]``, a parameter pair being bf16 (scale, offset). Byte j of a row of codes holds element
2j in its low nibble and 2j + 1 in its high one; an element's value is code * scale + offset.
"""
import math

import numpy as np
import torch

own = False

# ------------------------------------------------------------------------------------- cases
# append: `tokens` new tokens spread over `seqs` sequences, `heads` query and `kv_heads` key/value
# heads of `dim` elements, pages of `page` tokens, the first `rope` elements rotated.
# attend: `singles` sequences with one new token and `lo`..`hi` keys each, and `chunks` sequences
# with `chunk` new tokens and `history` keys before them; `window` 0 means every earlier key.


def _append(name, tokens, seqs, heads, kv_heads, dim, page, rope, interleaved=False):
    return {"name": name, "kind": "append", "tokens": tokens, "seqs": seqs, "heads": heads, "kv_heads": kv_heads,
            "dim": dim, "page": page, "rope": rope, "interleaved": interleaved}


def _attend(name, heads, kv_heads, dim, page, singles=0, lo=1, hi=1, chunks=0, chunk=1, history=0, window=0):
    return {"name": name, "kind": "attend", "heads": heads, "kv_heads": kv_heads, "dim": dim, "page": page,
            "singles": singles, "lo": lo, "hi": hi, "chunks": chunks, "chunk": chunk, "history": history,
            "window": window}


def listed():
    return [
        # one user, one token of a 4096-wide block with shared key/value heads: latency
        _append("append_one_token", 1, 1, 32, 8, 128, 16, 128),
        # a decode step of 64 users of the 4096-wide block with a key/value head per query head
        _append("append_batch_64", 64, 64, 32, 32, 128, 64, 128),
        # the mixed serving step: 64 decode tokens and a prefill chunk of 1024
        _append("append_step_1088", 1088, 65, 32, 32, 128, 128, 128),
        # prompts of the 8192-wide block, an odd number of tokens, interleaved pairs
        _append("append_prompts_12289", 12289, 5, 64, 8, 128, 64, 128, True),
        # one user, a short conversation: latency
        _attend("decode_one_333", 32, 8, 128, 16, singles=1, lo=333, hi=333),
        # the decode half of the mixed step: 64 users, ragged lengths, a key/value head per query head
        _attend("decode_64_ragged", 32, 32, 128, 64, singles=64, lo=100, hi=4096),
        # one user with a very long document: the work has to be split over its length
        _attend("decode_one_262143", 64, 8, 128, 128, singles=1, lo=262143, hi=262143),
        # a loaded server of the 8192-wide block: 128 users, lengths up to 8192
        _attend("decode_128_gqa", 64, 8, 128, 64, singles=128, lo=500, hi=8192),
        # four drafted tokens a sequence to verify, narrow heads, a sliding window
        _attend("verify_16x4_window", 32, 8, 64, 32, chunks=16, chunk=4, history=6001, window=4000),
        # a prefill chunk behind a cached prompt of odd length
        _attend("chunk_320_at_7901", 32, 8, 128, 16, chunks=1, chunk=320, history=7901),
        # the mixed serving step: 64 decode tokens and a chunk of 1024 with its own history
        _attend("mixed_64_1024", 32, 32, 128, 64, singles=64, lo=100, hi=2048, chunks=1, chunk=1024, history=1024),
        # a whole prompt at once: bound by the tensor cores
        _attend("prompt_8192", 32, 8, 128, 128, chunks=1, chunk=8192, history=0),
    ]


HEADS = [(32, 32), (32, 8), (64, 8), (16, 16), (28, 4), (10, 10), (12, 2), (8, 1)]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    heads, kv_heads = rng.choice(HEADS)
    dim, page = rng.choice([64, 128, 128]), rng.choice([16, 32, 48, 64, 128, 256])
    kind = rng.choice(["append", "append", "decode", "decode", "decode", "verify", "chunk", "chunk", "mixed"])
    if kind == "append":
        tokens = _log(rng, 1, 12289 * 80 // max(80, heads + 2 * kv_heads))
        rope = rng.choice([dim, dim, dim // 2])
        c = _append("", tokens, _log(rng, 1, min(tokens, 200)), heads, kv_heads, dim, page, rope, rng.random() < 0.3)
    else:
        room = 128 * 4346 * 8 * 128 // (kv_heads * dim)  # keys in all, as many bytes as the largest listed case
        window = _log(rng, 64, 4096) if rng.random() < 0.25 else 0
        if kind == "decode":
            n = _log(rng, 1, 256)
            hi = _log(rng, 1, max(1, min(200000, room // n)))
            c = _attend("", heads, kv_heads, dim, page, singles=n, lo=max(1, hi // rng.choice([1, 3, 20])), hi=hi, window=window)
        elif kind == "verify":
            n = _log(rng, 1, 64)
            c = _attend("", heads, kv_heads, dim, page, chunks=n, chunk=rng.randint(2, 8),
                        history=_log(rng, 1, max(1, min(30000, room // n // 2))), window=window)
        else:
            chunk = _log(rng, 16, 4096)
            history = _log(rng, 1, max(16, min(30000, (1 << 31) // (heads * chunk) - chunk, (1 << 30) // (heads * chunk) * 2)))
            n = 1 if heads * chunk * (chunk + history) > 1 << 28 else rng.randint(1, 4)
            c = _attend("", heads, kv_heads, dim, page, chunks=n, chunk=chunk, history=history, window=window)
            if kind == "mixed":
                hi = _log(rng, 16, 4096)
                c.update(singles=_log(rng, 1, 96), lo=max(1, hi // 8), hi=hi)
    del c["name"]
    return c


def _lengths(c):
    """New tokens and keys of each sequence, the ones with a single token first: ragged, and set by the case alone."""
    n = c["singles"]
    lens = [c["lo"] + int((c["hi"] - c["lo"]) * ((0.618034 * (i + 1)) % 1.0)) for i in range(n)]
    if n:
        lens[0] = c["hi"]
    return [1] * n + [c["chunk"]] * c["chunks"], lens + [c["history"] + c["chunk"]] * c["chunks"]


# ------------------------------------------------------------------------------------- inputs
def _rope_table(positions, rope):
    inv = 10000.0 ** (-torch.arange(0, rope, 2, device="cuda", dtype=torch.float64) / rope)
    a = torch.arange(positions, device="cuda", dtype=torch.float64)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float().contiguous()


def _fields(pool, page, dim):
    """Views of the cache: K codes, V codes (uint8 [page][head][block][16][D/2]) and the parameters (bf16 [..][16][2])."""
    b = pool.view(pool.shape[0], pool.shape[1], page // 16, 16 * (dim + 8))
    kc = b[..., :8 * dim].unflatten(-1, (16, dim // 2))
    vc = b[..., 8 * dim:16 * dim].unflatten(-1, (16, dim // 2))
    kp = b[..., 16 * dim:16 * dim + 64].view(torch.bfloat16).unflatten(-1, (16, 2))
    vp = b[..., 16 * dim + 64:].view(torch.bfloat16).unflatten(-1, (16, 2))
    return kc, vc, kp, vp


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _channels(g, *shape):
    return torch.exp(0.5 * _normal(g, *shape))  # channels of unequal size, as keys have them


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 13)
    rng = np.random.RandomState((int(seed) * 7919 + 13) % (1 << 32))
    hq, hk, dim, page = c["heads"], c["kv_heads"], c["dim"], c["page"]
    block = 16 * (dim + 8)
    s = {"case": dict(c)}
    if c["kind"] == "append":
        tokens, seqs = c["tokens"], c["seqs"]
        counts = [1] * (seqs - 1) + [tokens - (seqs - 1)] if seqs > 16 else [
            tokens // seqs + (i < tokens % seqs) for i in range(seqs)]  # decode tokens and a chunk, or several prompts
        first = rng.randint(0, 8192, size=seqs)
        pos = np.concatenate([f + np.arange(n) for f, n in zip(first, counts)])
        pages_of = [(f + n - 1) // page - f // page + 1 for f, n in zip(first, counts)]
        table = rng.permutation(sum(pages_of) + 7)  # the pages that the sequences touch, anywhere in the pool
        base = np.concatenate([[0], np.cumsum(pages_of)])
        slots = np.concatenate([table[base[i] + (f + np.arange(n)) // page - f // page] * page + (f + np.arange(n)) % page
                                for i, (f, n) in enumerate(zip(first, counts))])
        s["pool"] = torch.zeros(len(table), hk, page // 16 * block, dtype=torch.uint8, device="cuda")
        s["table"] = _rope_table(8192 + tokens, c["rope"])
        s["positions"] = torch.from_numpy(pos.astype(np.int64)).cuda()
        s["slots"] = torch.from_numpy(slots.astype(np.int64)).cuda()
        # the projections' output, one row of q, k and v heads a token
        qkv = _normal(g, tokens, hq + 2 * hk, dim)
        qkv[:, hq:hq + hk] *= _channels(g, hk, dim)
        qkv = qkv.bfloat16()
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
        s["q_out"] = torch.empty(tokens, hq, dim, dtype=torch.bfloat16, device="cuda")
        s["k_out"] = torch.empty(tokens, hk, dim, dtype=torch.bfloat16, device="cuda")
        s["v_out"] = torch.empty(tokens, hk, dim, dtype=torch.bfloat16, device="cuda")
    else:
        q_lens, kv_lens = _lengths(c)
        n_pages = [-(-x // page) for x in kv_lens]
        spare = 3
        table = np.zeros((len(kv_lens), max(n_pages)), np.int32)
        perm, at = rng.permutation(sum(n_pages) + spare).astype(np.int32), 0
        for i, n in enumerate(n_pages):
            table[i, :n] = perm[at:at + n]
            at += n
        pool = torch.empty(len(perm), hk, page // 16 * block, dtype=torch.uint8, device="cuda")
        kc, vc, kp, vp = _fields(pool, page, dim)
        scale = _channels(g, hk, 1, 1, dim)
        for p0 in range(0, len(perm), max(1, (1 << 27) // (hk * page * dim))):  # what earlier steps have cached
            p1 = min(len(perm), p0 + max(1, (1 << 27) // (hk * page * dim)))
            for codes, params, by in ((kc, kp, scale), (vc, vp, 1.0)):
                packed, pair = _quantise(_normal(g, p1 - p0, hk, page // 16, 16, dim) * by)
                codes[p0:p1], params[p0:p1] = packed, pair
        s["pool"] = pool
        s["page_table"] = torch.from_numpy(table).cuda()
        s["kv_lens"] = torch.tensor(kv_lens, dtype=torch.int32, device="cuda")
        s["q_starts"] = torch.tensor(np.concatenate([[0], np.cumsum(q_lens)]), dtype=torch.int32, device="cuda")
        s["max_q"] = max(q_lens)
        s["q"] = _normal(g, sum(q_lens), hq, dim).bfloat16()
        s["out"] = torch.empty(sum(q_lens), hq, dim, dtype=torch.bfloat16, device="cuda")
        s["scale"] = dim ** -0.5
    if own:  # the handle, made once for a model's layer and kept with its pool
        from quantized_linear_error_gb300 import spear
        s["cache"] = spear.SpearKVCache(hq, hk, dim, page, s["pool"], rope_table=s.get("table"),
                                        rope_interleaved=c.get("interleaved", False))
    return s


# ------------------------------------------------------------------------------------- plain forms
def _rotate(x, cos, sin, rope, interleaved):
    if interleaved:
        x1, x2 = x[..., 0:rope:2], x[..., 1:rope:2]
    else:
        x1, x2 = x[..., :rope // 2], x[..., rope // 2:rope]
    y = x.clone()
    r1, r2 = x1 * cos - x2 * sin, x2 * cos + x1 * sin
    if interleaved:
        y[..., 0:rope:2], y[..., 1:rope:2] = r1, r2
    else:
        y[..., :rope // 2], y[..., rope // 2:rope] = r1, r2
    return y


def _quantise(x):
    """Rows of fp32 values: packed codes uint8 [..., D/2] and (scale, offset) bf16 [..., 2]."""
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    scale = ((hi - lo) * (1.0 / 15.0)).bfloat16()
    scale = torch.where(scale.float() < 2.0 ** -126, torch.zeros_like(scale), scale)
    offset = lo.bfloat16()
    inv = torch.where(scale > 0, torch.reciprocal(scale.float()), torch.zeros_like(lo))
    code = torch.round((x - offset.float()) * inv).clamp(0, 15).to(torch.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), torch.cat([scale, offset], -1)


def _values(codes, params):
    """fp32 values of packed codes [..., D/2] with parameters bf16 [..., 2]."""
    p = params.float()
    code = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float()
    return code * p[..., :1] + p[..., 1:]


def _append_plain(s):
    c = s["case"]
    cs, half = s["table"][s["positions"]][:, None, :], c["rope"] // 2
    q = _rotate(s["q"].float(), cs[..., :half], cs[..., half:], c["rope"], c["interleaved"])
    k = _rotate(s["k"].float(), cs[..., :half], cs[..., half:], c["rope"], c["interleaved"])
    kc, vc, kp, vp = _fields(s["pool"], c["page"], c["dim"])
    page, at = s["slots"] // c["page"], s["slots"] % c["page"]
    block, row = at // 16, at % 16
    kc[page, :, block, row], kp[page, :, block, row] = _quantise(k)
    vc[page, :, block, row], vp[page, :, block, row] = _quantise(s["v"].float())
    return [q.bfloat16(), _values(kc[page, :, block, row], kp[page, :, block, row]).bfloat16(),
            _values(vc[page, :, block, row], vp[page, :, block, row]).bfloat16()]


def _attend_plain(s, first, last, n):
    """The sequences first..last - 1, each with n new tokens, as one padded batch: out fp32 [sequences * n][heads][dim]."""
    c = s["case"]
    hq, hk, dim, page = c["heads"], c["kv_heads"], c["dim"], c["page"]
    table = s["page_table"][first:last].long()
    seqs, lens = last - first, s["kv_lens"][first:last].long()
    row0 = first if n == 1 else c["singles"]
    q = s["q"][row0:row0 + seqs * n].float().view(seqs, n, hk, hq // hk, dim).permute(0, 2, 3, 1, 4) * s["scale"]
    q = q.reshape(seqs, hk, hq // hk * n, dim)
    kc, vc, kp, vp = (x[table].transpose(1, 2).flatten(2, 4) for x in _fields(s["pool"], page, dim))  # [seq][head][keys][..]
    scores = (q @ _values(kc, kp).transpose(-1, -2)).view(seqs, hk, hq // hk, n, -1)
    at = (lens[:, None] - n + torch.arange(n, device="cuda"))[:, None, None, :, None]
    j = torch.arange(scores.shape[-1], device="cuda")
    seen = (j <= at) & (j > at - c["window"]) if c["window"] else j <= at
    scores = scores.masked_fill(~seen, float("-inf"))
    p = torch.exp(scores - scores.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    out = p.flatten(2, 3) @ _values(vc, vp)
    return out.view(seqs, hk, hq // hk, n, dim).permute(0, 3, 1, 2, 4).reshape(seqs * n, hq, dim)


def run(state):
    s, c = state, state["case"]
    if c["kind"] == "append":
        if own:
            s["cache"].append(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["q_out"])
            s["cache"].read(s["slots"], s["k_out"], s["v_out"])
            return [s["q_out"], s["k_out"], s["v_out"]]
        return _append_plain(s)
    if own:
        return s["cache"].attention(s["q"], s["out"], s["page_table"], s["kv_lens"], s["q_starts"], s["max_q"],
                                    scale=s["scale"], window=c["window"])
    n = c["singles"]
    parts = [_attend_plain(s, 0, n, 1)] if n else []
    if c["chunks"]:
        parts.append(_attend_plain(s, n, n + c["chunks"], c["chunk"]))
    return torch.cat(parts).bfloat16()


# ------------------------------------------------------------------------------------- work
def _pairs(n, keys, window):
    """(query, key) pairs that n new tokens behind keys - n cached ones see, and the keys that any of them sees."""
    if not window:
        return n * (keys - n) + n * (n + 1) // 2, keys
    return sum(min(window, keys - n + i + 1) for i in range(n)), min(keys, window + n - 1)


def work(case):
    c = case
    hq, hk, dim = c["heads"], c["kv_heads"], c["dim"]
    if c["kind"] == "append":
        t = c["tokens"]
        # q, k, v in; rotated q, cached rows and the cached values out; a table row and two indices a token
        return {"bytes": t * ((hq + 2 * hk) * dim * 2 + hq * dim * 2 + hk * (dim + 8) + 2 * hk * dim * 2
                              + c["rope"] * 4 + 16),
                "flops": t * (3 * (hq + hk) * c["rope"] + 8 * hk * dim)}
    q_lens, kv_lens = _lengths(c)
    seen = [_pairs(n, k, c["window"]) for n, k in zip(q_lens, kv_lens)]
    return {"bytes": sum(k for _, k in seen) * hk * (dim + 8) + sum(q_lens) * hq * dim * 4,
            "flops": 4 * dim * hq * sum(p for p, _ in seen)}


# ------------------------------------------------------------------------------------- definition in 64 bits
def exact(case, seed):
    s, c = prepare(case, seed), case
    hq, hk, dim, page = c["heads"], c["kv_heads"], c["dim"], c["page"]
    if c["kind"] == "append":
        angle = s["table"].double()[s["positions"]]
        half = c["rope"] // 2
        first = torch.arange(half, device="cuda") * (2 if c["interleaved"] else 1)
        second = first + (1 if c["interleaved"] else half)

        def turned(x):
            x = x.double()
            y = x.clone()
            cos, sin = angle[:, None, :half], angle[:, None, half:]
            y[:, :, first] = x[:, :, first] * cos - x[:, :, second] * sin
            y[:, :, second] = x[:, :, first] * sin + x[:, :, second] * cos
            return y

        def held(x):
            lo, hi = x.min(-1, keepdim=True).values, x.max(-1, keepdim=True).values
            step, low = ((hi - lo) / 15).bfloat16().double(), lo.bfloat16().double()
            return ((x - low) / step).round().clamp(0, 15) * step + low

        return [turned(s["q"]), held(turned(s["k"])), held(s["v"].double())]
    q_lens, kv_lens = _lengths(c)
    raw = s["pool"].view(-1, hk, page // 16, 16 * (dim + 8))
    out, row, group = [], 0, hq // hk
    for i, (n, keys) in enumerate(zip(q_lens, kv_lens)):
        blocks = raw[s["page_table"][i, :-(-keys // page)].long()].transpose(0, 1).reshape(hk, -1, 16 * (dim + 8))

        def cached(h, codes_at, params_at):
            b = blocks[h, :, codes_at:codes_at + 8 * dim].reshape(-1, dim // 2)[:keys]
            par = blocks[h, :, params_at:params_at + 64].contiguous().view(torch.bfloat16).view(-1, 2)[:keys].double()
            code = torch.empty(keys, dim, dtype=torch.float64, device="cuda")
            code[:, 0::2], code[:, 1::2] = (b % 16).double(), (b // 16).double()
            return code * par[:, :1] + par[:, 1:]

        at = torch.arange(keys - n, keys, device="cuda")[:, None]
        j = torch.arange(keys, device="cuda")
        hidden = (j > at) if not c["window"] else (j > at) | (j <= at - c["window"])
        o = torch.empty(n, hq, dim, dtype=torch.float64, device="cuda")
        for h in range(hk):
            k, v = cached(h, 0, 16 * dim), cached(h, 8 * dim, 16 * dim + 64)
            for r in range(h * group, (h + 1) * group) if n > 64 else [slice(h * group, (h + 1) * group)]:
                q = s["q"][row:row + n, r].double()
                w = torch.einsum("n...d,jd->...nj", q, k) * s["scale"]
                w = torch.softmax(w.masked_fill(hidden, -math.inf), -1)
                o[:, r] = torch.einsum("...nj,jd->n...d", w, v)
        out.append(o)
        row += n
    return torch.cat(out)
