"""Measured cases of the 4-bit key/value cache: writing it and reading it back,
selecting its blocks for a step's queries, and attending over it.

The cache is paged, one page per block of ``block_size`` tokens, and each page
holds, per key/value head, tiles of 64 tokens:

  K codes [64 tokens][D/2 bytes] | V codes [32 token pairs][D bytes]
  | K (scale, zero) bf16 [64][D/64][2] | V (scale, zero) bf16 [64][D/64][2]

72 D bytes in all. Channel c of a key sits in byte ((c%32)/8)(D/8) + (c/32)4 +
(c%8)/2 of its token's row, in the low four bits for even c. Channel c of the
value of token r sits in byte (((c%32)/4) ^ 2((r/2)%4))(D/8) + (c/32)4 +
(r%2)2 + (c%4)/2 of its pair's row. A value is zero + scale * code.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # a step of generation: one new token of each of 64 sequences, written behind caches of differing lengths
        dict(name="write step", op="write", B=64, T=1, H=16, H_kv=4, D=128, block_size=64, length=2048, ragged=True,
             topk=0, dtype="bf16"),
        # prompts of a padded batch in float32, each starting inside a page
        dict(name="write prompts f32", op="write", B=8, T=1531, H=16, H_kv=16, D=64, block_size=64, length=4000,
             ragged=True, topk=0, dtype="f32"),
        # one long prompt, the benchmark's 131072 tokens of 16 heads
        dict(name="write long prompt", op="write", B=1, T=131072, H=16, H_kv=16, D=128, block_size=128, length=131072,
             ragged=False, topk=0, dtype="bf16"),
        # selection for one sequence of 8192 tokens: the smallest call
        dict(name="topk one sequence", op="topk", B=1, T=1, H=16, H_kv=4, D=64, block_size=64, length=8192,
             ragged=False, topk=38, dtype="bf16"),
        # a serving batch at the benchmark's length: 1024 blocks, 15% kept
        dict(name="topk batch", op="topk", B=32, T=1, H=16, H_kv=4, D=128, block_size=128, length=131072, ragged=True,
             topk=153, dtype="bf16"),
        # one sequence of a million tokens: 4096 blocks, several new tokens
        dict(name="topk million", op="topk", B=1, T=3, H=8, H_kv=8, D=128, block_size=256, length=1048576,
             ragged=False, topk=614, dtype="bf16"),
        # the smallest call of the attention: one sequence, a few pages, latency counts
        dict(name="attn short", op="attn", B=1, T=1, H=16, H_kv=4, D=128, block_size=64, length=397, ragged=False,
             topk=0, dtype="bf16"),
        # a batch of chats of differing lengths, dense
        dict(name="attn ragged batch", op="attn", B=48, T=1, H=16, H_kv=2, D=64, block_size=64, length=8192,
             ragged=True, topk=0, dtype="bf16"),
        # long dense contexts
        dict(name="attn dense 32k", op="attn", B=16, T=1, H=16, H_kv=4, D=128, block_size=128, length=32768,
             ragged=False, topk=0, dtype="bf16"),
        # the benchmark's length with 15% of the blocks kept
        dict(name="attn sparse 128k", op="attn", B=16, T=1, H=16, H_kv=4, D=128, block_size=128, length=131072,
             ragged=True, topk=153, dtype="bf16"),
        # several new tokens at once (drafted tokens to verify), a padded batch
        dict(name="attn drafts", op="attn", B=8, T=5, H=16, H_kv=2, D=128, block_size=64, length=16384, ragged=True,
             topk=0, dtype="bf16"),
        # float32 queries, every head with its own keys
        dict(name="attn f32", op="attn", B=5, T=1, H=12, H_kv=12, D=64, block_size=64, length=6001, ragged=True,
             topk=0, dtype="f32"),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("write", "topk", "attn", "attn"))
    D = rng.choice((64, 128))
    bs = rng.choice((64, 128, 256))
    hkv = rng.choice((1, 2, 3, 4, 8, 16))
    group = rng.choice((1, 2, 3, 4, 5, 8, 16))
    dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
    ragged = rng.random() < 0.6
    if op == "write":
        B = _log(rng, 1, 64)
        length = _log(rng, 1, max(1, (1 << 26) // (B * hkv * D)))
        T = 1 if rng.random() < 0.4 else _log(rng, 1, length)
        topk = 0
    else:
        B = _log(rng, 1, 64)
        # up to the blocks or tokens of the largest listed case of the operator
        most = (bs << 16 if op == "topk" else 1 << 21) // (B * hkv)
        length = _log(rng, 1, max(1, min(1 << 20, most)))
        T = 1 if rng.random() < 0.6 else rng.randint(2, 9)
        length = max(length, T)
        blocks = -(-length // bs)
        topk = max(1, int(blocks * rng.uniform(0.05, 0.6))) if op == "topk" or rng.random() < 0.5 else 0
        if topk:
            ragged = ragged and blocks > 1
    return dict(op=op, B=B, T=T, H=hkv * group, H_kv=hkv, D=D, block_size=bs, length=length, ragged=ragged, topk=topk,
                dtype=dtype)


# ------------------------------------------------------------------ the cache's layout


def _places(D, device):
    """Byte and shift of each channel of a key in its row [D], and of each
    (token, channel) of the values in a tile's V codes [64, D]."""
    c = torch.arange(D, device=device)
    r = torch.arange(64, device=device)[:, None]
    k_byte = (c % 32) // 8 * (D // 8) + c // 32 * 4 + c % 8 // 2
    v_byte = r // 2 * D + ((c % 32 // 4) ^ (2 * (r // 2 % 4))) * (D // 8) + c // 32 * 4 + r % 2 * 2 + c % 4 // 2
    return k_byte, v_byte, (c % 2 * 4).to(torch.uint8)


def _values(tiles, D):
    """Keys and values [..., 64, D] in float32 of cache tiles [..., 72 D] (uint8)."""
    k_byte, v_byte, shift = _places(D, tiles.device)
    lead = tiles.shape[:-1]
    k = tiles[..., : 32 * D].reshape(*lead, 64, D // 2)[..., k_byte]
    v = tiles[..., 32 * D: 64 * D][..., v_byte.reshape(-1)].reshape(*lead, 64, D)
    sz = tiles[..., 64 * D:].contiguous().view(torch.bfloat16).reshape(*lead, 2, 64, D // 64, 1, 2).float()
    out = []
    for n, b in enumerate((k, v)):
        code = ((b >> shift) & 15).float().reshape(*lead, 64, D // 64, 64)
        out.append((sz[..., n, :, :, :, 1] + sz[..., n, :, :, :, 0] * code).reshape(*lead, 64, D))
    return out


def _quantise(x):
    """Codes (uint8), scale and zero (bf16, one for each group of 64 channels) of x [..., D] in float32."""
    g = x.reshape(*x.shape[:-1], -1, 64)
    zero = g.amin(-1, keepdim=True).bfloat16()
    scale = ((g.amax(-1, keepdim=True) - zero.float()) * (1 / 15)).bfloat16()
    scale = torch.where(scale.float() < 2.0 ** -126, torch.zeros_like(scale), scale)
    inverse = torch.where(scale == 0, torch.zeros_like(scale).double(), 1 / scale.double()).float()
    code = torch.round((g - zero.float()) * inverse).clamp(0, 15)
    return code.to(torch.uint8).reshape(x.shape), scale.squeeze(-1), zero.squeeze(-1)


def _tiles(k, v):
    """Cache tiles [n, 72 D] of keys and values [n, 64, D]."""
    n, _, D = k.shape
    k_byte, v_byte, shift = _places(D, k.device)
    (kc, ks, kz), (vc, vs, vz) = _quantise(k), _quantise(v)
    pair = lambda c: c[..., 0::2] | c[..., 1::2] << 4  # noqa: E731
    kb = torch.empty(n, 64, D // 2, dtype=torch.uint8, device=k.device)
    kb[..., k_byte[0::2]] = pair(kc)
    vb = torch.empty(n, 32 * D, dtype=torch.uint8, device=k.device)
    vb[:, v_byte[:, 0::2].reshape(-1)] = pair(vc).reshape(n, -1)
    sz = [torch.stack((s, z), -1).reshape(n, -1).view(torch.uint8) for s, z in ((ks, kz), (vs, vz))]
    return torch.cat((kb.reshape(n, -1), vb, *sz), 1)


# ------------------------------------------------------------------ inputs


def _keys_values(gen, n, D):
    """Keys with an offset of their own in every channel, and values: [n, D] each."""
    offset = torch.randn(D, generator=gen, device="cuda")
    return (torch.randn(n, D, generator=gen, device="cuda") + offset, torch.randn(n, D, generator=gen, device="cuda"))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    B, T, H, Hk, D, bs = (case[n] for n in ("B", "T", "H", "H_kv", "D", "block_size"))
    dtype, length = _DT[case["dtype"]], max(case["length"], T)
    if case["ragged"]:  # lengths between T and the longest, and padded rows: fewer new tokens, none for the last of four
        u = torch.rand(B, generator=gen, device="cuda")
        start = ((length - T) * (0.1 + 0.9 * u)).to(torch.int32)
        count = torch.randint(1, T + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)
        count[3::4] = 0
        count[0] = T
        start[0] = length - T
    else:
        start = torch.full((B,), length - T, dtype=torch.int32, device="cuda")
        count = torch.full((B,), T, dtype=torch.int32, device="cuda")
    P = -(-length // bs)
    total = start + count
    used = (total + bs - 1) // bs
    ids = torch.randperm(B * P + 5, generator=gen, device="cuda")[: B * P].to(torch.int32).reshape(B, P)
    table = torch.where(torch.arange(P, device="cuda")[None] < used[:, None], ids, torch.full_like(ids, -1))
    pages = B * P + 5
    s = dict(case=dict(case), start=start, count=count, table=table)
    if case["op"] != "write":
        s["q"] = torch.randn(B, T, H, D, generator=gen, device="cuda").mul_(1.5).to(dtype)
    if case["op"] in ("write", "topk"):
        if case["op"] == "topk":  # sums of keys around a mean of the block's own
            s["k_sum"] = torch.randn(pages, Hk, D, generator=gen, device="cuda") * bs
        else:
            s["k_sum"] = torch.zeros(pages, Hk, D, device="cuda")
    if case["op"] in ("write", "attn"):  # tiles drawn from 2048 made of keys and values, so that they hold real codes
        n = pages * Hk * (bs // 64)
        k, v = _keys_values(gen, 64 * 2048, D)
        made = _tiles(k.reshape(-1, 64, D), v.reshape(-1, 64, D))
        at = torch.randint(0, made.shape[0], (n,), generator=gen, device="cuda")
        s["cache"] = made[at].reshape(pages, Hk, bs // 64, 72 * D)
    if case["op"] == "write":
        k, v = _keys_values(gen, B * T * Hk, D)
        s["k"], s["v"] = (x.to(dtype).reshape(B, T, Hk, D) for x in (k, v))
        s["k_out"], s["v_out"] = torch.zeros_like(s["k"]), torch.zeros_like(s["v"])
    if case["op"] == "attn":
        s["idx"] = None
        if case["topk"]:  # some of the sequence's blocks, the newest among them, ascending, padded with -1
            score = torch.rand(B, Hk, P, generator=gen, device="cuda")
            j = torch.arange(P, device="cuda")
            score = torch.where(j >= used[:, None, None] - 1, 2.0, score)
            score = torch.where(j >= used[:, None, None], -1.0, score)
            best, idx = score.topk(min(case["topk"], P), -1)
            idx = torch.where(best < 0, P, idx).sort(-1).values
            s["idx"] = torch.where(idx == P, -1, idx).to(torch.int32).contiguous()
        s["out"] = torch.zeros_like(s["q"])
    return s


# ------------------------------------------------------------------ one pass


def run(s):
    c = s["case"]
    if own:
        import block_sparse_attention_19_b200 as bsa

        if c["op"] == "write":
            bsa.bsa_cache_write(s["k"], s["v"], s["cache"], s["k_sum"], s["table"], s["start"], c["block_size"],
                                count=s["count"])
            bsa.bsa_cache_read(s["cache"], s["table"], s["start"], c["T"], c["block_size"], count=s["count"],
                               k_out=s["k_out"], v_out=s["v_out"])
            return dict(k=s["k_out"], v=s["v_out"], k_sum=s["k_sum"])
        if c["op"] == "topk":
            return dict(idx=bsa.bsa_cache_block_topk(s["q"], s["k_sum"], s["table"], s["start"], c["topk"],
                                                     c["block_size"], count=s["count"]))
        return dict(o=bsa.bsa_cache_attn(s["q"], s["cache"], s["table"], s["start"], c["block_size"], idx=s["idx"],
                                         count=s["count"], out=s["out"]))
    return {"write": _write, "topk": _topk, "attn": _attn}[c["op"]](s)


def _write(s):
    c = s["case"]
    B, T, Hk, D, bs = c["B"], c["T"], c["H_kv"], c["D"], c["block_size"]
    dev = s["k"].device
    pos = s["start"][:, None].long() + torch.arange(T, device=dev)
    new = torch.arange(T, device=dev) < s["count"][:, None]
    block = (pos // bs).clamp(max=s["table"].shape[1] - 1)
    page = torch.gather(s["table"].long(), 1, block)
    b, t = torch.nonzero(new & (page >= 0), as_tuple=True)
    page, row = page[b, t], pos[b, t] % bs
    tile = (page[:, None] * Hk + torch.arange(Hk, device=dev)) * (bs // 64) + row[:, None] // 64  # [n, Hk]
    r = row % 64
    k_byte, v_byte, _ = _places(D, dev)
    flat = s["cache"].view(-1)
    at = tile[..., None] * (72 * D)
    half = at + 64 * D + (r * (D // 16))[:, None, None]
    places = (((r * (D // 2))[:, None] + k_byte[0::2], half), (32 * D + v_byte[:, 0::2][r], half + 4 * D))
    for x, (codes, scales) in ((s["k"], places[0]), (s["v"], places[1])):
        code, scale, zero = _quantise(x[b, t].float())
        flat[at + codes[:, None]] = code[..., 0::2] | code[..., 1::2] << 4
        flat[scales + torch.arange(D // 16, device=dev)] = torch.stack((scale, zero), -1).flatten(-2).view(torch.uint8)
    # the touched pages' sums, over their tokens up to the last one written
    slots = s["start"][:, None].long() // bs + torch.arange((T + bs - 2) // bs + 1, device=dev)
    end = (s["start"] + s["count"])[:, None].long()
    some = (slots * bs < end) & (s["count"][:, None] > 0) & (slots < s["table"].shape[1])
    page = torch.gather(s["table"].long(), 1, slots.clamp(max=s["table"].shape[1] - 1))
    some &= page >= 0
    rows = (end - slots * bs)[some].clamp(max=bs)
    page = page[some]
    keys = _values(s["cache"][page], D)[0].reshape(-1, Hk, bs, D)
    keys = torch.where((torch.arange(bs, device=dev) < rows[:, None])[:, None, :, None], keys, 0.0)
    s["k_sum"][page] = keys.sum(2, dtype=torch.float64).float()
    # and the new rows read back
    for out, (codes, scales) in ((s["k_out"], places[0]), (s["v_out"], places[1])):
        code = flat[at + codes[:, None]]
        code = torch.stack((code & 15, code >> 4), -1).float().reshape(*tile.shape, D // 64, 64)
        scale, zero = flat[scales + torch.arange(D // 16, device=dev)].view(torch.bfloat16).float().unflatten(
            -1, (D // 64, 2)).unbind(-1)
        out[b, t] = (zero[..., None] + scale[..., None] * code).reshape(*tile.shape, D).to(out.dtype)
    return dict(k=s["k_out"], v=s["v_out"], k_sum=s["k_sum"])


def _topk(s):
    c = s["case"]
    B, T, H, Hk, D, bs = (c[n] for n in ("B", "T", "H", "H_kv", "D", "block_size"))
    P, dev = s["table"].shape[1], s["q"].device
    new = (torch.arange(T, device=dev) < s["count"][:, None])[:, :, None, None]
    q = torch.where(new, s["q"].float(), 0.0).reshape(B, T, Hk, H // Hk, D).sum((1, 3), dtype=torch.float64)
    j = torch.arange(P, device=dev)
    tokens = ((s["start"] + s["count"])[:, None].long() - j * bs).clamp(0, bs)  # of each block
    there = (tokens > 0) & (s["table"] >= 0)
    sums = s["k_sum"][s["table"].long().clamp(min=0)].double()  # [B, P, Hk, D]
    score = (torch.matmul(sums.permute(0, 2, 1, 3), q[..., None]).squeeze(-1) / tokens.clamp(min=1)[:, None]).float()
    score = torch.where(there[:, None], score, -math.inf)
    k = c["topk"]
    order = score.sort(dim=-1, stable=True, descending=True).indices[..., :k]
    there = there[:, None].expand(-1, Hk, -1).gather(-1, order)
    order = torch.where(there, order, P).sort(-1).values
    return dict(idx=torch.where(order == P, -1, order).to(torch.int32))


def _attn(s):
    c = s["case"]
    B, T, H, Hk, D, bs = (c[n] for n in ("B", "T", "H", "H_kv", "D", "block_size"))
    P, dev = s["table"].shape[1], s["q"].device
    idx = s["idx"] if s["idx"] is not None else torch.arange(P, device=dev, dtype=torch.int32).expand(B, Hk, P)
    at = idx.long().clamp(min=0)
    page = s["table"].long()[:, None].expand(-1, Hk, -1).gather(2, at)
    pos = torch.where((idx >= 0) & (page >= 0), at * bs, 1 << 40)[..., None] + torch.arange(bs, device=dev)
    pos = pos.flatten(2)  # [B, Hk, n]
    k, v = _values(s["cache"][page.clamp(min=0), torch.arange(Hk, device=dev)[None, :, None]], D)
    k, v = k.reshape(B, Hk, -1, D), v.reshape(B, Hk, -1, D)
    q = s["q"].float().reshape(B, T, Hk, H // Hk, D).permute(0, 2, 1, 3, 4).reshape(B, Hk, -1, D)
    x = torch.matmul(q, k.transpose(-1, -2)) * D ** -0.5
    own_pos = (s["start"][:, None].long() + torch.arange(T, device=dev)).repeat_interleave(H // Hk, 1)
    seen = pos[:, :, None] <= own_pos[:, None, :, None]
    x = torch.where(seen, x, -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
    o = torch.matmul(p, v) / p.sum(-1, keepdim=True).clamp(min=1e-30)
    o = o.reshape(B, Hk, T, H // Hk, D).permute(0, 2, 1, 3, 4).reshape(B, T, H, D)
    new = (torch.arange(T, device=dev) < s["count"][:, None])[:, :, None, None]
    return dict(o=torch.where(new, o.to(s["out"].dtype), s["out"]))


# ------------------------------------------------------------------ work and the definition in 64 bits


def _sizes(case):
    """Expected start and count over the sequences, as prepare draws them."""
    B, T, length = case["B"], case["T"], max(case["length"], case["T"])
    if not case["ragged"]:
        return [(length - T, T)] * B
    some = [(length - T, T)] + [((length - T) * 0.55, 0 if b % 4 == 3 else (T + 1) / 2) for b in range(1, B)]
    return some


def work(case):
    T, H, Hk, D, bs = (case[n] for n in ("T", "H", "H_kv", "D", "block_size"))
    es = 2 if case["dtype"] == "bf16" else 4
    sizes, P = _sizes(case), -(-max(case["length"], T) // bs)
    row = D // 2 + D // 16  # a token's codes, scale and zero, for one head, keys or values
    if case["op"] == "write":
        n = sum(c for _, c in sizes) * Hk
        touched = sum((a % bs + c + bs - 1) // bs for a, c in sizes if c) * Hk
        return {"bytes": n * (2 * D * es + 2 * row) + n * (2 * row + 2 * D * es) + touched * D * 4, "flops": n * D * 20}
    new = sum(c for _, c in sizes)
    if case["op"] == "topk":
        n = sum(math.ceil((a + c) / bs) for a, c in sizes) * Hk
        return {"bytes": n * D * 4 + new * H * D * es + case["B"] * (Hk * case["topk"] + P) * 4, "flops": 2 * n * D}
    kept = min(case["topk"] or P, P) * bs
    n = sum(min(a + c, kept) for a, c in sizes if c) * Hk
    f = sum(min(a + c, kept) * c for a, c in sizes) * H * D * 4
    return {"bytes": n * 2 * row + 2 * new * H * D * es, "flops": f}


def _words(tiles, D):
    """Keys and values in float64 of cache tiles [..., 72 D], from 32-bit words of eight codes."""
    lead = tiles.shape[:-1]
    w = tiles.contiguous().view(torch.int32)
    dev = tiles.device
    eight = torch.arange(0, 32, 4, device=dev, dtype=torch.int32)
    k = (w[..., : 8 * D].reshape(*lead, 64, 4, D // 32, 1) >> eight) & 15  # token, eight channels of 32, 32 channels
    k = k.transpose(-2, -3).reshape(*lead, 64, D)
    v = w[..., 8 * D: 16 * D].reshape(*lead, 8, 4, 8, D // 32)  # eight tokens, pair, slot, 32 channels
    v = torch.stack([v[..., p, [g ^ (2 * p) for g in range(8)], :] for p in range(4)], -3)
    v = ((v[..., None] >> eight) & 15).unflatten(-1, (2, 4))  # ..., 8, pair, four channels, 32, which of the pair, channel
    n = len(lead)
    v = v.permute(*range(n), n, n + 1, n + 4, n + 3, n + 2, n + 5).reshape(*lead, 64, D)
    sz = tiles[..., 64 * D:].contiguous().view(torch.bfloat16).double().reshape(*lead, 2, 64, D // 64, 2)
    sz = sz.repeat_interleave(64, -2)
    return [sz[..., i, :, :, 1] + sz[..., i, :, :, 0] * x for i, x in enumerate((k, v))]


def _held(x):
    """What the cache holds of x [..., D], in float64: each group of 64 channels on sixteen steps from its lowest
    value; the steps themselves are float32 arithmetic by definition."""
    out = []
    for g in x.double().split(64, -1):
        lo, hi = g.min(-1).values, g.max(-1).values
        z = lo.bfloat16().double()
        sc = ((hi - z).float().double() * torch.tensor(1 / 15).item()).float().bfloat16().double()
        sc[sc < 2.0 ** -126] = 0
        inv = torch.zeros_like(sc)
        inv[sc > 0] = (1 / sc[sc > 0]).float().double()
        d = (g - z[..., None]).float().double()
        code = (d * inv[..., None]).float().double().round().clip(0, 15)
        out.append(z[..., None] + sc[..., None] * code)
    return torch.cat(out, -1)


def exact(case, seed):
    s = prepare(case, seed)
    T, H, Hk, D, bs = (case[n] for n in ("T", "H", "H_kv", "D", "block_size"))
    start, count, table = s["start"].tolist(), s["count"].tolist(), s["table"].tolist()
    if case["op"] == "write":
        k_out, v_out = (torch.zeros(s["k"].shape, dtype=torch.float64, device="cuda") for _ in "kv")
        k_sum = s["k_sum"].double()
        for b, (a, n) in enumerate(zip(start, count)):
            if not n:
                continue
            k_out[b, :n], v_out[b, :n] = _held(s["k"][b, :n]), _held(s["v"][b, :n])
            first, last = a // bs, (a + n - 1) // bs
            page = torch.tensor(table[b][first: last + 1], device="cuda")
            lead = a - first * bs
            older = _words(s["cache"][page[0]], D)[0].reshape(Hk, bs, D)[:, :lead]
            keys = torch.cat((older, k_out[b, :n].transpose(0, 1)), 1)
            keys = torch.cat((keys, keys.new_zeros(Hk, (last - first + 1) * bs - keys.shape[1], D)), 1)
            k_sum[page] = keys.reshape(Hk, -1, bs, D).sum(2).transpose(0, 1)
        return dict(k=k_out, v=v_out, k_sum=k_sum)
    if case["op"] == "topk":
        idx = torch.full((case["B"], Hk, case["topk"]), -1, dtype=torch.int32)
        for b, (a, n) in enumerate(zip(start, count)):
            blocks = -(-(a + n) // bs)
            if not blocks:
                continue
            q = s["q"][b, :n].double().reshape(n, Hk, H // Hk, D).sum((0, 2))
            tokens = [bs] * (blocks - 1) + [a + n - (blocks - 1) * bs]
            sums = s["k_sum"][torch.tensor(table[b][:blocks], device="cuda")].double()
            score = (torch.einsum("hd,jhd->hj", q, sums) / torch.tensor(tokens, device="cuda")).float().tolist()
            for h in range(Hk):
                best = sorted(range(blocks), key=lambda j: (-score[h][j], j))[: case["topk"]]
                idx[b, h, : len(best)] = torch.tensor(sorted(best), dtype=torch.int32)
        return dict(idx=idx)
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for b, (a, n) in enumerate(zip(start, count)):
        if not n:
            continue
        for h in range(Hk):
            blocks = range(-(-(a + n) // bs)) if s["idx"] is None else [j for j in s["idx"][b, h].tolist() if j >= 0]
            page = torch.tensor([table[b][j] for j in blocks], device="cuda")
            pos = torch.tensor(list(blocks), device="cuda")[:, None] * bs + torch.arange(bs, device="cuda")
            k, v = (x.reshape(-1, D) for x in _words(s["cache"][page, h], D))
            heads = slice(h * (H // Hk), (h + 1) * (H // Hk))
            x = torch.einsum("tgd,nd->tgn", s["q"][b, :n, heads].double(), k) / math.sqrt(D)
            hidden = pos.reshape(-1)[None] > (a + torch.arange(n, device="cuda"))[:, None]
            x.masked_fill_(hidden[:, None], -math.inf)
            o[b, :n, heads] = torch.einsum("tgn,nd->tgd", x.softmax(-1).nan_to_num(0.0), v)
    return dict(o=o)
