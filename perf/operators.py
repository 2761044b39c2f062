"""Cases for the 4-bit paged cache: writing, reading back, and attention over it.

A pool holds, per (layer, page, KV head), blocks of 16 tokens. A block is one
record of bytes: K codes, V codes, K parameters, V parameters.

- K codes: 16 token rows of D/2 bytes. A row is four chunks t of D/32 little-endian
  32-bit words w; nibble 4*el + 2*jj + eh of the word holds channel
  16*(2*w + jj) + 4*t + 2*eh + el.
- V codes: two halves of 8 tokens, each [g 8][pair 4][parity 2][D/16 bytes]: token
  2*pair + parity of the half, channels g*D/8 + 0, 1, ... from the low nibble up.
- parameters: [16 tokens][D/group][scale, minimum] in the cache's 16-bit type.

A value is scale * code + minimum; a scale has seven significant bits. A batch says where its rows are: `table`
[B, pages a sequence] (page ids), `kv_len` [B] (tokens a sequence has, the
batch's own rows included) and `start` [B + 1] (row offsets); a sequence's rows are
its last ones.
"""
import math

import torch

own = False

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


def _case(name, op, dtype="fp16", layers=1, seqs=1, heads=32, kv_heads=8, dim=128, group=64, page=64, rows=(1, 1), lens=(4096, 4096),
          fused=False, window=0, lse=False, f32=False):
    c = {"op": op, "dtype": dtype, "layers": layers, "seqs": seqs, "heads": heads, "kv_heads": kv_heads, "dim": dim, "group": group, "page": page,
         "rows_lo": rows[0], "rows_hi": rows[1], "len_lo": lens[0], "len_hi": lens[1], "fused": fused, "window": window, "lse": lse, "f32": f32}
    return {"name": name, **c} if name else c


def listed():
    return [
        # one decoding step of a small batch stores its new tokens: latency
        _case("write_step_8", "write", seqs=8, page=16, lens=(100, 4000)),
        # the step of a large batch, K and V sliced out of the fused projection's rows
        _case("write_step_256", "write", "bf16", seqs=256, page=16, lens=(1, 2000), fused=True),
        # a restored 4096-token prefix of 32 layers goes into the pool
        _case("write_prefix", "write", layers=32, rows=(4096, 4096), lens=(4096, 4096)),
        # prompts of odd lengths behind what their sequences already hold, small heads, small groups
        _case("write_ragged", "write", "bf16", seqs=16, kv_heads=16, dim=64, group=32, page=32, rows=(3, 2011), lens=(2011, 5003)),
        # a few short contexts read back in binary32, wide heads
        _case("read_short", "read", "bf16", seqs=3, kv_heads=4, dim=256, group=128, page=16, rows=(201, 1013), lens=(201, 1013), f32=True),
        # contexts read back for an attention that wants 16 bits
        _case("read_long", "read", seqs=8, rows=(5000, 32768), lens=(5000, 32768)),
        # one user's next token: latency
        _case("step_1", "attend", page=16, lens=(4096, 4096)),
        # a serving batch's next tokens, lengths spread
        _case("step_64", "attend", "bf16", seqs=64, lens=(700, 16384), lse=True),
        # long contexts, eight query heads a KV head
        _case("step_long", "attend", seqs=4, heads=64, page=128, lens=(81920, 81920)),
        # drafted tokens checked at once, as many KV heads as query heads, a sliding window
        _case("draft_16", "attend", "bf16", seqs=16, heads=16, kv_heads=16, dim=64, group=32, page=32, rows=(1, 7), lens=(301, 9001), window=4096),
        # the rest of a prompt behind a restored prefix
        _case("chunk_512", "attend", "bf16", rows=(512, 512), lens=(8704, 8704), lse=True),
        # a long prompt's chunk, the largest
        _case("chunk_4096", "attend", rows=(4096, 4096), lens=(32768, 32768)),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    dim = rng.choice([64, 128, 128, 256])
    shape = {"dtype": rng.choice(["fp16", "bf16"]), "dim": dim, "group": rng.choice([g for g in (32, 64, 128) if g <= dim]),
             "page": rng.choice([16, 32, 64, 128])}
    op = rng.choice(["write", "read", "attend", "attend", "attend"])
    kv = rng.choice([1, 2, 4, 8])
    if op in ("write", "read"):
        seqs = _spread(rng, 1, 64)
        layers = _spread(rng, 1, 16)
        most = max(1, min(32768, (1 << 27) // (seqs * layers * kv * dim)))
        hi = _spread(rng, 1, most)
        lo = rng.randint(1, hi)
        past = 0 if op == "read" else rng.randint(0, 3000)
        return _case(None, op, layers=layers, seqs=seqs, heads=4 * kv, kv_heads=kv, rows=(lo, hi), lens=(lo + past, hi + past),
                     fused=op == "write" and layers == 1 and rng.random() < 0.5, f32=op == "read" and rng.random() < 0.3, **shape)
    heads = kv * rng.choice([1, 2, 4, 5, 8])
    window = rng.choice([0, 0, 0, 512, 4096])
    lse = rng.random() < 0.5
    if rng.random() < 0.65:  # next tokens, or a few drafted ones
        seqs = _spread(rng, 1, 128)
        rows = (1, 1) if rng.random() < 0.6 else (1, rng.randint(2, 8))
        hi = _spread(rng, 16, max(16, min(65536, (1 << 30) // (seqs * kv * dim))))
        return _case(None, op, seqs=seqs, heads=heads, kv_heads=kv, rows=rows, lens=(rng.randint(8, max(8, hi)), max(8, hi)), window=window, lse=lse, **shape)
    seqs = rng.choice([1, 1, 2, 3])  # prompts, or chunks of them
    hi = _spread(rng, 17, 2048)
    past = rng.choice([0, rng.randint(1, 8000)])
    return _case(None, op, seqs=seqs, heads=heads, kv_heads=kv, rows=(max(1, hi // 2), hi), lens=(hi + past, hi + past), window=window, lse=lse, **shape)


def _between(lo, hi, n, turn):
    """n whole numbers between lo and hi, the last one hi, the others spread."""
    return [hi if b == n - 1 else lo + int((hi - lo) * ((b * 0.6180339887 + turn) % 1.0)) for b in range(n)]


def _lengths(case):
    n = case["seqs"]
    lens = _between(case["len_lo"], case["len_hi"], n, 0.37)
    rows = lens if case["op"] == "read" else [min(r, k) for r, k in zip(_between(case["rows_lo"], case["rows_hi"], n, 0.71), lens)]
    return lens, rows


def work(case):
    lens, rows = _lengths(case)
    n, H, D, w = sum(rows), case["kv_heads"], case["dim"], case["window"]
    stored = H * (D + 8 * (D // case["group"]))  # bytes a token of one layer
    if case["op"] == "write":
        return {"bytes": case["layers"] * n * (4 * H * D + stored + 4 * H * D), "flops": 0}
    if case["op"] == "read":
        return {"bytes": case["layers"] * n * (stored + (8 if case["f32"] else 4) * H * D), "flops": 0}
    seen = pairs = 0
    for k, r in zip(lens, rows):
        seen += k if not w else min(k, w + r - 1)
        at = range(k - r + 1, k + 1)  # keys a row sees without a window
        pairs += sum(at) if not w else sum(min(a, w) for a in at)
    return {"bytes": seen * stored + n * case["heads"] * (4 * D + (4 if case["lse"] else 0)), "flops": 4 * D * case["heads"] * pairs}


def _quantised(x, group, dtype):
    """Codes (uint8) and [scale, minimum] (in `dtype`) of binary32 x [..., D]."""
    g = x.unflatten(-1, (-1, group))
    lo, hi = g.amin(-1, keepdim=True), g.amax(-1, keepdim=True)
    s = ((hi - lo) / 15).view(torch.int32)
    s = ((s + 0x10000) & ~0x1FFFF).view(torch.float32).to(dtype).float()  # seven significant bits
    s = torch.where(torch.isfinite(hi - lo), s, torch.nan)
    lo = torch.where(torch.isfinite(s), lo, torch.nan)
    c = torch.where(s > 0, torch.round((g - lo) / s).clamp(0, 15), 0.0)
    return c.to(torch.uint8).flatten(-2), torch.cat([s, lo], -1).to(dtype)


def _k_bytes(c):
    """Codes [..., D] of K rows as their D/2 bytes."""
    D = c.shape[-1]
    c = c.unflatten(-1, (D // 32, 2, 4, 2, 2))  # w, jj, t, eh, el
    c = c.permute(*range(c.dim() - 5), -3, -5, -1, -4, -2)  # t, w, el, jj, eh
    return (c[..., 0] + 16 * c[..., 1]).flatten(-4)


def _k_codes(b):
    D = 2 * b.shape[-1]
    c = torch.stack([b & 15, b >> 4], -1).unflatten(-2, (4, D // 32, 2, 2))  # t, w, el, jj, eh
    return c.permute(*range(c.dim() - 5), -4, -2, -5, -1, -3).flatten(-5)


def _v_bytes(c):
    return c[..., 0::2] + 16 * c[..., 1::2]


def _v_codes(b):
    return torch.stack([b & 15, b >> 4], -1).flatten(-2)


def _parts(pool, case):
    """Views of the pool's bytes: K codes [..., 2, 8, D/2], V codes [..., 2, 8, 4, 2, D/16], parameters [..., 16, 4 D/group] of K and of V."""
    D = case["dim"]
    p = 64 * (D // case["group"])
    return (pool[..., :8 * D].unflatten(-1, (2, 8, D // 2)), pool[..., 8 * D:16 * D].unflatten(-1, (2, 8, 4, 2, D // 16)),
            pool[..., 16 * D:16 * D + p].unflatten(-1, (16, -1)), pool[..., 16 * D + p:].unflatten(-1, (16, -1)))


def _fill(pool, case, g):
    """Every slot of one layer's pages holds a quantised token: keys with channels of different spread and offset, a few of them large."""
    H, D, P = case["kv_heads"], case["dim"], case["page"]
    dtype = TYPES[case["dtype"]]
    kc, vc, kp, vp = _parts(pool, case)
    sk, mk, sv, _ = _spreads(case, g)
    step = max(1, (1 << 27) // (P * H * D))
    for a in range(0, pool.shape[0], step):
        n = min(step, pool.shape[0] - a)
        x = torch.randn(n, H, P // 16, 16, D, device="cuda", generator=g)
        c, p = _quantised((x * sk[:, None, None] + mk[:, None, None]).to(dtype).float(), case["group"], dtype)
        kc[a:a + n] = _k_bytes(c).unflatten(-2, (2, 8))
        kp[a:a + n] = p.contiguous().view(torch.uint8).flatten(-2)
        x = torch.randn(n, H, P // 16, 16, D, device="cuda", generator=g)
        c, p = _quantised((x * sv[:, None, None]).to(dtype).float(), case["group"], dtype)
        vc[a:a + n] = _v_bytes(c).unflatten(-2, (2, 4, 2)).unflatten(-1, (8, -1)).permute(0, 1, 2, 3, 6, 4, 5, 7)
        vp[a:a + n] = p.contiguous().view(torch.uint8).flatten(-2)


def _spreads(case, g):
    H, D = case["kv_heads"], case["dim"]
    sk = torch.exp(0.5 * torch.randn(H, D, device="cuda", generator=g))
    sk = torch.where(torch.rand(H, D, device="cuda", generator=g) < 0.02, 4 * sk, sk)
    mk = 0.7 * sk * torch.randn(H, D, device="cuda", generator=g)
    sv = 0.6 * torch.exp(0.3 * torch.randn(H, D, device="cuda", generator=g))
    return sk, mk, sv, torch.zeros_like(sv)


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    lens, rows = _lengths(case)
    H, D, P, L = case["kv_heads"], case["dim"], case["page"], case["layers"]
    dtype = TYPES[case["dtype"]]
    need = [-(-k // P) for k in lens]
    pages = sum(need) + 3
    order = torch.randperm(pages, device="cuda", generator=g).to(torch.int32)
    table = torch.zeros(len(lens), max(need), dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    state = {"case": case, "rows": sum(rows), "max_rows": max(rows), "table": table, "kv_len": torch.tensor(lens, dtype=torch.int32, device="cuda"),
             "start": None if rows == [1] * len(rows) else torch.tensor([0] + rows, device="cuda").cumsum(0).to(torch.int32)}
    pool = torch.zeros(L, pages, H, P // 16, 16 * D + 128 * (D // case["group"]), dtype=torch.uint8, device="cuda")
    state["pool"] = pool
    if case["op"] == "write":
        spreads = _spreads(case, g)
        wide = (case["heads"] + 2 * H) * D
        for name, (s, m), at in (("k", spreads[:2], case["heads"] * D), ("v", spreads[2:], (case["heads"] + H) * D)):
            x = torch.randn(L, sum(rows), H, D, device="cuda", generator=g)
            x = (x * s + m).to(dtype).reshape(L, -1, H * D)
            if case["fused"]:
                if name == "k":
                    state["qkv"] = torch.zeros(L, sum(rows), wide, dtype=dtype, device="cuda")
                state["qkv"][..., at:at + H * D] = x
                x = state["qkv"][..., at:at + H * D]
            state[name] = x
        return state
    for layer in range(L):
        _fill(pool[layer], case, g)
    if case["op"] == "attend":
        state["q"] = torch.randn(sum(rows), case["heads"], D, device="cuda", generator=g).to(dtype)
    return state


def _row_places(state):
    """Per row of the batch: its sequence, its position in it, its page and its place in the page."""
    lens, start, P = state["kv_len"].long(), state["start"], state["case"]["page"]
    n = torch.arange(state["rows"], device="cuda")
    if start is None:
        b, at = n, lens - 1
    else:
        b = torch.searchsorted(start.long(), n, right=True) - 1
        at = lens[b] - (start[b + 1].long() - n)
    return b, at, state["table"][b, at // P].long(), at % P


def _values(codes, params, group, dtype):
    p = params.contiguous().view(dtype).unflatten(-1, (-1, 2)).float()
    return (codes.unflatten(-1, (-1, group)).float() * p[..., :1] + p[..., 1:]).flatten(-2)


def _plain_write(state):
    case = state["case"]
    dtype, H, D = TYPES[case["dtype"]], case["kv_heads"], case["dim"]
    _, _, page, slot = _row_places(state)
    blk, half, r = slot // 16, slot // 8 % 2, slot % 8
    kc, vc, kp, vp = _parts(state["pool"], case)
    c, p = _quantised(state["k"].unflatten(-1, (H, D)).float().transpose(0, 1), case["group"], dtype)
    kc[:, page, :, blk, half, r] = _k_bytes(c)
    kp[:, page, :, blk, slot % 16] = p.contiguous().view(torch.uint8).flatten(-2)
    c, p = _quantised(state["v"].unflatten(-1, (H, D)).float().transpose(0, 1), case["group"], dtype)
    vc[:, page, :, blk, half, :, r // 2, r % 2] = _v_bytes(c).unflatten(-1, (8, -1))
    vp[:, page, :, blk, slot % 16] = p.contiguous().view(torch.uint8).flatten(-2)


def _plain_read(state):
    case = state["case"]
    dtype = TYPES[case["dtype"]]
    out = torch.float32 if case["f32"] else dtype
    _, _, page, slot = _row_places(state)
    blk, half, r = slot // 16, slot // 8 % 2, slot % 8
    kc, vc, kp, vp = _parts(state["pool"], case)
    k = _values(_k_codes(kc[:, page, :, blk, half, r]), kp[:, page, :, blk, slot % 16], case["group"], dtype)
    v = _values(_v_codes(vc[:, page, :, blk, half, :, r // 2, r % 2].flatten(-2)), vp[:, page, :, blk, slot % 16], case["group"], dtype)
    most = torch.finfo(out).max
    return {"k": k.clamp(-most, most).to(out).transpose(0, 1).flatten(-2), "v": v.clamp(-most, most).to(out).transpose(0, 1).flatten(-2)}


def _plain_attend(state):
    case, q = state["case"], state["q"]
    dtype, H, D, P = TYPES[case["dtype"]], case["kv_heads"], case["dim"], case["page"]
    B, R = case["seqs"], case["heads"] // H
    T = state["table"].shape[1] * P
    kc, vc, kp, vp = _parts(state["pool"][0], case)
    at = state["table"].long()
    # [B, pages, H, blocks, ...] -> [B, H, T, D]
    flat = lambda x: x.permute(0, 2, 1, 3, *range(4, x.dim())).flatten(2, -2)  # noqa: E731
    k = flat(_values(_k_codes(kc[at].flatten(-3, -2)), kp[at], case["group"], dtype))
    v = flat(_values(_v_codes(vc[at].permute(0, 1, 2, 3, 4, 6, 7, 5, 8).flatten(-2).flatten(4, 6)), vp[at], case["group"], dtype))
    b, pos, _, _ = _row_places(state)
    n = state["max_rows"]
    row = pos - (state["kv_len"].long()[b] - n)  # last rows at the end
    padded = torch.zeros(B, n, H, R, D, device="cuda")
    padded[b, row] = q.float().unflatten(1, (H, R))
    padded = padded.permute(0, 2, 3, 1, 4).flatten(2, 3)  # [B, H, R * n, D]
    s = (padded @ k.transpose(-1, -2)).unflatten(2, (R, n)) * D ** -0.5
    i = (state["kv_len"].long()[:, None] - n + torch.arange(n, device="cuda"))[:, None, None, :, None]
    j = torch.arange(T, device="cuda")
    seen = (j <= i) & (j > i - case["window"]) if case["window"] else j <= i
    s.masked_fill_(~seen, -math.inf)
    top = s.amax(-1, keepdim=True).clamp_min(-3e38)
    s = s.sub_(top).exp_()
    total = s.sum(-1, keepdim=True)
    v = v.masked_fill(~(j < state["kv_len"][:, None])[:, None, :, None], 0.0)
    o = (s.flatten(2, 3) @ v).unflatten(2, (R, n)) / total.clamp_min(1e-37)
    pick = lambda x: x.permute(0, 3, 1, 2, 4).flatten(2, 3)[b, row]  # noqa: E731  [N, heads, ...]
    out = {"out": pick(o).to(dtype)}
    if case["lse"]:
        out["lse"] = pick(top + total.log()).squeeze(-1)
    return out


def _own(state):
    """The cache and the batch as a program keeps them."""
    if "cache" not in state:
        from kv_cache_compression_cg_gb300 import cache4
        c = state["case"]
        state["cache"] = cache4.Cache4(c["layers"], state["pool"].shape[1], c["page"], c["kv_heads"], c["dim"], group=c["group"], dtype=TYPES[c["dtype"]],
                                       pool=state["pool"])
        state["batch"] = cache4.Batch4(state["table"], state["kv_len"], state["start"], rows=state["rows"], max_rows=state["max_rows"])
    return state["cache"], state["batch"]


def run(state):
    op = state["case"]["op"]
    if not own:
        if op == "attend":
            return _plain_attend(state)
        if op == "write":
            _plain_write(state)
        return _plain_read(state)
    cache, batch = _own(state)
    if op == "attend":
        if state["case"]["lse"]:
            out, lse = cache.attend(state["q"], batch, window=state["case"]["window"], return_lse=True)
            return {"out": out, "lse": lse}
        return {"out": cache.attend(state["q"], batch, window=state["case"]["window"])}
    if op == "write":
        cache.write_layers(state["k"], state["v"], batch)
    k, v = cache.read_layers(batch, dtype=torch.float32 if state["case"]["f32"] else None)
    return {"k": k, "v": v}


def _places(case):
    """Where a block's record holds each (token of 16, channel): byte and shift of K codes, of V codes, and the byte of the group's parameters."""
    D, G = case["dim"], case["group"]
    t, d = torch.arange(16, device="cuda")[:, None], torch.arange(D, device="cuda")[None, :]
    word, in16 = d // 32, d % 16
    nib = 4 * (in16 % 2) + 2 * (d // 16 % 2) + in16 // 2 % 2
    k = t * (D // 2) + (in16 // 4) * (D // 8) + word * 4 + nib // 2
    g, i = d // (D // 8), d % (D // 8)
    v = 8 * D + (t // 8) * 4 * D + g * (D // 2) + (t % 8) * (D // 16) + i // 2
    p = 16 * D + (t * (D // G) + d // G) * 4
    return k, (4 * (nib % 2)).expand(16, D), v, (4 * (i % 2)).expand(16, D), p


def _stored64(state, layer, pages):
    """K and V [pages, H, P, D] of these pages in 64 bits, taken byte by byte from the records."""
    case = state["case"]
    dtype = TYPES[case["dtype"]]
    rec = state["pool"][layer][pages]
    kb, ks, vb, vs, pb = _places(case)
    got = []
    for b, sh, base in ((kb, ks, 0), (vb, vs, 64 * (case["dim"] // case["group"]))):
        code = ((rec[..., b].int() >> sh) & 15).double()
        two = lambda at: (rec[..., at].to(torch.int32) | (rec[..., at + 1].to(torch.int32) << 8)).to(torch.int16).view(dtype).double()  # noqa: E731
        got.append((code * two(pb + base) + two(pb + base + 2)).flatten(2, 3))
    return got


def exact(case, seed):
    state = prepare(case, seed)
    lens, rows = _lengths(case)
    H, D, P, G = case["kv_heads"], case["dim"], case["page"], case["group"]
    if case["op"] == "write":
        dtype, out = TYPES[case["dtype"]], {}
        for name in ("k", "v"):
            whole = []
            for x in state[name]:
                x = x.double().reshape(-1, H, D // G, G)
                low = x.min(-1, keepdim=True).values
                fraction, power = torch.frexp((x.max(-1, keepdim=True).values - low) / 15)
                s = torch.ldexp(torch.floor(fraction * 128 + 0.5) / 128, power).to(dtype).double()
                code = torch.where(s > 0, ((x - low) / torch.where(s > 0, s, 1.0)).round().clamp(0, 15), 0.0)
                whole.append((code * s + low).reshape(-1, H * D))
            out[name] = torch.stack(whole)
        return out
    k_all, v_all, o_all, l_all = [], [], [], []
    if case["op"] == "read":
        for layer in range(case["layers"]):
            ks, vs = [], []
            for b, n in enumerate(lens):
                k, v = _stored64(state, layer, state["table"][b, :-(-n // P)].long())
                ks.append(k.transpose(1, 2).reshape(-1, H * D)[:n])
                vs.append(v.transpose(1, 2).reshape(-1, H * D)[:n])
            k_all.append(torch.cat(ks))
            v_all.append(torch.cat(vs))
        return {"k": torch.stack(k_all), "v": torch.stack(v_all)}
    at, R, w = 0, case["heads"] // H, case["window"]
    for b, (n, r) in enumerate(zip(lens, rows)):
        k, v = _stored64(state, 0, state["table"][b, :-(-n // P)].long())
        k, v = (x.transpose(0, 1).reshape(H, -1, D)[:, :n] for x in (k, v))
        o = torch.empty(r, case["heads"], D, dtype=torch.float64, device="cuda")
        lse = torch.empty(r, case["heads"], dtype=torch.float64, device="cuda")
        i, j = torch.arange(n - r, n, device="cuda")[:, None], torch.arange(n, device="cuda")[None, :]
        hidden = (j > i) | (j <= i - w) if w else j > i
        for h in range(case["heads"]):
            s = state["q"][at:at + r, h].double() @ k[h // R].T / math.sqrt(D)
            s.masked_fill_(hidden, -math.inf)
            lse[:, h] = torch.logsumexp(s, -1)
            o[:, h] = torch.exp(s - lse[:, h, None]) @ v[h // R]
        o_all.append(o)
        l_all.append(lse)
        at += r
    return {"out": torch.cat(o_all), "lse": torch.cat(l_all)} if case["lse"] else {"out": torch.cat(o_all)}
