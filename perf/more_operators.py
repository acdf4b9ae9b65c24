"""What is measured of the operators for long contexts: a paged key/value cache in 4 bits, what reads it, and the
eviction of the tokens that attention looks at least.

  append   new keys are turned by their positions, keys and values are brought to 4 bits and written into the cache; the
           values that the cache then holds for these tokens come back (q8k_kv4_append, q8k_kv4_read)
  attend   softmax attention of new tokens over the 4-bit cache, from one token a sequence to whole prompts (qattend_kv4)
  weights  what each cached token gets of the new tokens' attention, added up over the query heads of its key head, over a
           cache of 8 or 4 bits (qattend_weights)
  evict    of each sequence and key head the tokens of the largest weights are kept, with the first and the last ones,
           and moved to the front of other pages; what these hold comes back (q8k_kv_evict, and the caches' reads)

`own` chooses between the library's calls and the plain torch forms.
"""
import math

import torch

own = False

PAGE = 64  # tokens of a cache page
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # a decode batch in a padded (graph-captured) step: some of its rows stand for no sequence
        dict(name="append_batch_61", op="append", tokens=61, pad=3, kv_heads=8, dim=128, dtype="f32", rot=128,
             pairs="adjacent"),
        # prompts entering the cache, partial rotation, odd count
        dict(name="append_prompt_8191", op="append", tokens=8191, pad=0, kv_heads=8, dim=128, dtype="bf16", rot=64,
             pairs="half"),
        # one conversation's next token after a short prompt
        dict(name="attend_1x513", op="attend", batch=1, q=1, len=513, ragged=False, q_heads=32, kv_heads=8, dim=128,
             dtype="f32", window=0, rot=128, pairs="half"),
        # a decode batch of conversations of many lengths
        dict(name="attend_16x8191", op="attend", batch=16, q=1, len=8191, ragged=True, q_heads=32, kv_heads=8, dim=128,
             dtype="f32", window=0, rot=128, pairs="adjacent"),
        # decode over long documents, what the 4 bits are for
        dict(name="attend_8x65537", op="attend", batch=8, q=1, len=65537, ragged=False, q_heads=32, kv_heads=8, dim=128,
             dtype="bf16", window=0, rot=0, pairs="half"),
        # a prompt of 512 tokens from its start
        dict(name="attend_prompt_512", op="attend", batch=1, q=512, len=512, ragged=False, q_heads=32, kv_heads=8,
             dim=128, dtype="f32", window=0, rot=128, pairs="half"),
        # chunks of long prompts, over what of them the cache already holds
        dict(name="attend_chunk_3x1000_16001", op="attend", batch=3, q=1000, len=16001, ragged=True, q_heads=32,
             kv_heads=4, dim=128, dtype="bf16", window=0, rot=128, pairs="half"),
        # each decode step adds to what the cached tokens have gathered
        dict(name="weights_16x8191", op="weights", bits=8, batch=16, q=1, len=8191, ragged=True, q_heads=32, kv_heads=8,
             dim=128, dtype="f32", window=0, rot=128, pairs="adjacent", keep=1.0),
        # the last 64 tokens of long prompts say what of these is worth keeping
        dict(name="weights_last64_4x16001", op="weights", bits=4, batch=4, q=64, len=16001, ragged=True, q_heads=32,
             kv_heads=8, dim=128, dtype="bf16", window=0, rot=128, pairs="half", keep=0.0),
        # every token of a chunk counts, older ones less
        dict(name="weights_chunk_2x1000_8001", op="weights", bits=4, batch=2, q=1000, len=8001, ragged=False, q_heads=32,
             kv_heads=4, dim=128, dtype="bf16", window=0, rot=128, pairs="half", keep=0.9),
        # one conversation over its budget by a few tokens
        dict(name="evict_1x2111", op="evict", bits=4, batch=1, len=2111, ragged=False, kv_heads=8, dim=128, budget=2048,
             first=4, last=256),
        # long prompts cut to a quarter of the longest, some of them short enough to stay whole
        dict(name="evict_16x16001", op="evict", bits=8, batch=16, len=16001, ragged=True, kv_heads=8, dim=128,
             budget=4000, first=4, last=500),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "attend", "weights", "weights", "evict"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    bits = rng.choice([8, 4])
    dim = rng.choice([64, 128, 128, 256])
    rot = rng.choice([0, dim, dim, dim // 2])
    pairs = rng.choice(["half", "adjacent"])
    if op == "append":
        kv_heads = rng.choice([1, 2, 4, 8, 16])
        tokens = _log(rng, 1, min(8191, 8191 * 1024 // (kv_heads * dim)))
        return dict(op=op, tokens=tokens, pad=rng.choice([0, 0, 1, 7]), kv_heads=kv_heads, dim=dim, dtype=dtype,
                    rot=rot, pairs=pairs)
    kv_heads = rng.choice([1, 2, 4, 8])
    if op == "evict":
        batch = _log(rng, 1, 16)
        length = _log(rng, 100, min(65537, 16 * 16001 * 8 * 128 // (batch * kv_heads * dim)))
        budget = max(1, int(length * rng.uniform(0.1, 1.0)))
        budget = min(budget, max(1, 16 * 4000 * 8 * 128 // (batch * kv_heads * dim)))
        last = int(budget * rng.uniform(0.0, 0.5))
        return dict(op=op, bits=bits, batch=batch, len=length, ragged=rng.random() < 0.7, kv_heads=kv_heads, dim=dim,
                    budget=budget, first=min(rng.choice([0, 1, 4]), budget - last), last=last)
    q_heads = kv_heads * rng.choice([1, 2, 4, 6, 8])
    few = rng.random() < 0.6
    if few:  # decode, or a few drafted tokens
        q = rng.choice([1, 1, 1, 2, 5, 8])
        batch = _log(rng, 1, 64)
        top = (8 * 65537 * 8 * 128) // (batch * kv_heads * dim)
        length = _log(rng, max(q, 16), max(64, min(65537, top)))
    else:  # prompts and chunks of them
        q = _log(rng, 16, 1000)
        batch = rng.choice([1, 1, 2, 3, 5])
        # cost (and the plain form's score matrix) at most about half of attend_chunk_3x1000_16001's
        top = (500 * 16001 * 32 * 3) // (batch * q * q_heads * max(1, dim // 128))
        length = _log(rng, q, max(q, min(16001, top)))
    case = dict(op=op, batch=batch, q=q, len=length, ragged=rng.random() < 0.7, q_heads=q_heads, kv_heads=kv_heads,
                dim=dim, dtype=dtype, window=rng.choice([0, 0, 0, max(1, length // 3)]), rot=rot, pairs=pairs)
    if op == "weights":
        case.update(bits=bits, keep=rng.choice([0.0, 0.9, 1.0]))
    return case


def _lengths(case):
    """(new tokens, cached tokens with the new ones) of each sequence: the first has the most of both, the others
    spread evenly below that where the case is ragged."""
    got = []
    for b in range(case["batch"]):
        f = (b * 0.6180339887498949) % 1.0 if case["ragged"] else 0.0
        new = max(1, int(case.get("q", 1) * (1.0 - 0.9 * f)))
        got.append((new, max(new, int(case["len"] * (1.0 - 0.9 * f)))))
    return got


# ---------------------------------------------------------------- the caches
# One record for each page and key head.  A token's bytes of a record lie at places that only its number in the page
# decides; `_map(bits, dim)` is their table [64 tokens][bytes], in the order
#   8 bits: the key's codes, the value's codes [dim each], the key's scale, the value's [4 each]
#   4 bits: the key's codes (two of them a byte, as below), the value's [dim/2 each], the factors of the key's groups of
#           32 values, those of the value's [dim/32 each], the key's scale, the value's [4 each]
# In 4 bits a value is (code * factor) * scale, code + 8 in four bits and a factor in eight: those of an fp16 whose bits
# are factor << 6.  Of a key, sixteen values from 16 h on make two words of eight, value j of a word at the bits from
# 4 (j/2 + 4 (j%2)) + 2 on, round the word's end.  Of a value vector, those at 32 e + c and 32 e + 16 + c share a byte,
# the first in the low half.
_MAPS = {}


def _record_bytes(bits, dim):
    return 2 * PAGE * dim + 8 * PAGE if bits == 8 else 68 * dim + 512


def _map(bits, dim):
    if (bits, dim) in _MAPS:
        return _MAPS[bits, dim]
    t = torch.arange(PAGE)[:, None]
    i = torch.arange(dim)[None]
    if bits == 8:
        place = ((t >> 2) & 3) << 4 | (t >> 5) << 3 | ((t >> 4) & 1) << 2 | (t & 3)
        k = (i >> 6) * 4096 + t * 64 + (i & 63)
        v = PAGE * dim + i * PAGE + place
        end = 2 * PAGE * dim
        parts = [k, v]
    else:
        place = ((t >> 2) & 3) << 4 | (t >> 5) << 3 | ((t >> 4) & 1) << 2 | (t & 1) << 1 | ((t >> 1) & 1)
        n = dim // 64
        # bytes of a key, eight for each sixteen values 64 s + 16 h
        y = torch.arange(dim // 2)[None]
        s, h, b = (y >> 3) // 4, (y >> 3) % 4, y & 7
        piece = (t // 16) * n + s
        k = (piece >> 1) * 1024 + (t % 16 * 4 + h) * 16 + (piece & 1) * 8 + b
        e, c = y // 16, y % 16
        v = 32 * dim + e * 1024 + c * 64 + place
        g = torch.arange(dim // 32)[None]
        kf = 64 * dim + (t % 16 * 2 + g % 2) * (dim // 16) + (t // 16) * n + g // 2
        vf = 66 * dim + g * 64 + place
        end = 68 * dim
        parts = [k, v, kf, vf]
    four = torch.arange(4)[None]
    _MAPS[bits, dim] = torch.cat(parts + [end + 4 * t + four, end + 256 + 4 * t + four], 1).cuda()
    return _MAPS[bits, dim]


def _quantise8(x):
    most = x.abs().amax(-1, keepdim=True)
    codes = torch.where(most > 0, torch.round(x * (127.0 / most)).clamp(-127, 127), torch.zeros_like(x))
    return codes.to(torch.int8).view(torch.uint8), (most / 127.0).squeeze(-1)


def _factor(f):
    """Factors as they lie in the cache -> their values."""
    return (f.to(torch.int16) << 6).view(torch.float16).float()


def _quantise4(x):
    """Codes (as float, [..., dim]), the bytes of the groups' factors [..., dim/32] and scales [...] of the last axis.
    Scale: the largest magnitude / 7.  A group's factor: the least that is not below its largest magnitude / the row's."""
    groups = x.unflatten(-1, (-1, 32))
    top = groups.abs().amax(-1)
    most = top.amax(-1, keepdim=True)
    scale = most / torch.full_like(most, 7.0)
    r = torch.where(most > 0, top / most, torch.zeros_like(top))
    bits = r.view(torch.int32)
    byte = torch.where(r >= 2.0 ** -14, ((bits + 0x7ffff) >> 19) - (112 << 4), (r * 2.0 ** 18).ceil().int())
    step = (_factor(byte) * scale)[..., None]
    codes = torch.where(byte[..., None] > 0, torch.round(groups * (1.0 / step)), torch.zeros_like(groups))
    return codes.clamp(-7, 7).flatten(-2), byte.to(torch.uint8), scale.squeeze(-1)


def _token_bytes(bits, k, v):
    """The bytes [..., as _map's] that stand for fp32 keys and values [..., dim]."""
    lead = k.shape[:-1]
    f32 = lambda s: s.unsqueeze(-1).contiguous().view(torch.uint8)  # noqa: E731
    if bits == 8:
        (kc, ks), (vc, vs) = _quantise8(k), _quantise8(v)
        return torch.cat([kc, vc, f32(ks), f32(vs)], -1)
    (kc, kf, ks), (vc, vf, vs) = _quantise4(k), _quantise4(v)
    u = (kc + 8).to(torch.int64).unflatten(-1, (-1, 8))
    j = torch.arange(8, device=k.device)
    word = (u << (4 * (j // 2 + 4 * (j % 2)) + 2)).sum(-1)
    word = word + (word >> 32)
    kb = (word[..., None] >> 8 * j[:4]).to(torch.uint8).reshape(*lead, -1)
    u = (vc + 8).to(torch.uint8).unflatten(-1, (-1, 2, 16))
    vb = (u[..., 0, :] | (u[..., 1, :] << 4)).flatten(-2)
    return torch.cat([kb, vb, kf, vf, f32(ks), f32(vs)], -1)


def _held(bits, raw, dim):
    """fp32 keys and values [..., dim] that the bytes [..., as _map's] stand for."""
    f32 = lambda b: b.contiguous().view(torch.float32)  # noqa: E731
    if bits == 8:
        k, v = raw[..., :dim].view(torch.int8).float(), raw[..., dim: 2 * dim].view(torch.int8).float()
        return k * f32(raw[..., 2 * dim: 2 * dim + 4]), v * f32(raw[..., 2 * dim + 4:])
    n, g = dim // 2, dim // 32
    lead = raw.shape[:-1]
    word = raw[..., :n].contiguous().view(torch.int32)[..., None]
    j = torch.arange(8, device=raw.device, dtype=torch.int32)
    at = (4 * (j // 2 + 4 * (j % 2)) + 2) % 32
    # the last code lies round the word's end (a shift to the right keeps the sign, which the mask takes off)
    kc = torch.where(j < 7, word >> at, (word >> 30 & 3) | word << 2).bitwise_and(15).float() - 8
    b = raw[..., n: 2 * n].unflatten(-1, (-1, 16))
    vc = torch.stack([b & 15, b >> 4], -2).float() - 8
    kf, vf = _factor(raw[..., 2 * n: 2 * n + g]), _factor(raw[..., 2 * n + g: 2 * n + 2 * g])
    s = 2 * n + 2 * g
    k = (kc.reshape(*lead, g, 32) * kf[..., None]).flatten(-2) * f32(raw[..., s: s + 4])
    v = (vc.reshape(*lead, g, 32) * vf[..., None]).flatten(-2) * f32(raw[..., s + 4:])
    return k, v


def _rope_table(positions, rot):
    """[positions][rot]: the cosines, then the sines, of the angles p / 10000^(2i/rot), from 64 bits."""
    i = torch.arange(rot // 2, device="cuda", dtype=torch.float64)
    a = torch.arange(positions, device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (-2.0 * i / rot)
    return torch.cat([a.cos(), a.sin()], 1).float()


def _rotate(x, table, pos, rot, pairs):
    """x [tokens, heads, dim], its first `rot` values turned by the angles of `pos`."""
    if not rot:
        return x
    row = table.to(x.dtype)[pos.long()][:, None, :]
    c, s = row[..., : rot // 2], row[..., rot // 2:]
    if pairs == "half":
        a, b = x[..., : rot // 2], x[..., rot // 2: rot]
        y = torch.cat([a * c - b * s, a * s + b * c], -1)
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)
    return torch.cat([y, x[..., rot:]], -1)


# ---------------------------------------------------------------- prepare
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _prepare_append(case, g):
    T, H, D, dt = case["tokens"], case["kv_heads"], case["dim"], TYPES[case["dtype"]]
    n = T + case["pad"]
    # keys and values as the projection leaves them: side by side in one row (here behind 4 query heads a key head)
    row = torch.randn(n, 6 * H, D, device="cuda", generator=g)
    row *= torch.rand(n, 6 * H, 1, device="cuda", generator=g) * 3 + 0.2
    row[..., ::17] *= 4  # a few channels stand out
    row = row.to(dt)
    # pages handed out in no order; tokens run on from the middle of the first page
    count = (T + 37 + PAGE - 1) // PAGE + 5
    order = torch.randperm(count, device="cuda", generator=g)
    at = torch.arange(T, device="cuda") + 37
    slots = torch.cat([order[at // PAGE] * PAGE + at % PAGE, torch.full((case["pad"],), -1, device="cuda")]).int()
    pos = torch.cat([at, torch.zeros(case["pad"], device="cuda", dtype=at.dtype)]).int()
    # one page more than the cache has: the plain form's place for rows that stand for no token
    cache = torch.zeros(count + 1, H, _record_bytes(4, D), dtype=torch.uint8, device="cuda")
    return dict(case=case, row=row, k=row[:, 4 * H: 5 * H], v=row[:, 5 * H:], slots=slots, pos=pos, n=n, cache=cache,
                pages=count, table=_rope_table(T + 37, case["rot"]) if case["rot"] else None,
                k_out=torch.zeros(n, H, D, device="cuda", dtype=torch.bfloat16),
                v_out=torch.zeros(n, H, D, device="cuda", dtype=torch.bfloat16))


def _filled_cache(bits, count, H, D, g):
    cache = torch.empty(count, H, _record_bytes(bits, D), dtype=torch.uint8, device="cuda")
    # keys whose products with the queries spread as trained heads' do: a few channels stand out
    lift = torch.rand(H, 1, D, device="cuda", generator=g) ** 4 * 2 + 0.5
    at = _map(bits, D).flatten()
    for p in range(0, count, 128):
        m = min(count, p + 128) - p
        k = torch.randn(m, H, PAGE, D, device="cuda", generator=g) * lift
        v = torch.randn(m, H, PAGE, D, device="cuda", generator=g)
        cache[p: p + m][..., at] = _token_bytes(bits, k, v).flatten(-2)
    return cache


def _page_table(seqs, g):
    per = [(l + PAGE - 1) // PAGE for _, l in seqs]
    count = sum(per)
    order = torch.randperm(count, device="cuda", generator=g).int()
    pages = torch.full((len(per), max(per)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(per):
        pages[b, :n] = order[at: at + n]
        at += n
    return count, pages


def _prepare_queries(case, g):
    B, Hq, H, D = case["batch"], case["q_heads"], case["kv_heads"], case["dim"]
    seqs = _lengths(case)
    count, pages = _page_table(seqs, g)
    starts = [0]
    for new, _ in seqs:
        starts.append(starts[-1] + new)
    Tq = starts[-1]
    row = (torch.randn(Tq, Hq + 2 * H, D, device="cuda", generator=g) * 1.5).to(TYPES[case["dtype"]])
    lens = torch.tensor([l for _, l in seqs], dtype=torch.int32, device="cuda")
    cu_q = torch.tensor(starts, dtype=torch.int32, device="cuda")
    seq_of = torch.repeat_interleave(torch.arange(B, device="cuda"), cu_q.diff().long())
    index = torch.arange(Tq, device="cuda") - cu_q.long()[seq_of]
    pos = (lens.long()[seq_of] - cu_q.diff().long()[seq_of] + index).int()
    return dict(case=case, bits=case.get("bits", 4), q=row[:, :Hq], row=row, pages=pages, lens=lens, cu_q=cu_q, pos=pos,
                Tq=Tq, seq_of=seq_of, index=index, max_q=max(n for n, _ in seqs), max_len=max(l for _, l in seqs),
                count=count, cache=_filled_cache(case.get("bits", 4), count, H, D, g),
                table=_rope_table(case["len"], case["rot"]) if case["rot"] else None, scale=1.0 / math.sqrt(D),
                out=torch.zeros(Tq, Hq, D, device="cuda", dtype=row.dtype), lse=torch.zeros(Tq, Hq, device="cuda"))


def _prepare_weights(case, g):
    s = _prepare_queries(case, g)
    # what the attention before left: each row's log of its sum (of the same inputs, rounded to 32 bits)
    s["lse"] = _lse64(s).float()
    shape = (case["batch"], case["kv_heads"], s["max_len"] + 5)
    s["old"] = torch.rand(shape, device="cuda", generator=g) ** 8 * 50 if case["keep"] else None
    s["weights"] = torch.zeros(shape, device="cuda")
    return s


def _prepare_evict(case, g):
    B, H, D, n = case["batch"], case["kv_heads"], case["dim"], case["budget"]
    seqs = _lengths(case)
    count, pages = _page_table(seqs, g)
    most = max(l for _, l in seqs)
    # what attention left: most tokens gathered next to nothing, a few much
    weights = torch.rand(B, H, most + 3, device="cuda", generator=g) ** 12 * 100
    out_per = (n + PAGE - 1) // PAGE
    out_pages = torch.randperm(B * out_per, device="cuda", generator=g).int().view(B, out_per) + count
    lens = torch.tensor([l for _, l in seqs], dtype=torch.int32, device="cuda")
    cache = torch.zeros(count + B * out_per, H, _record_bytes(case["bits"], D), dtype=torch.uint8, device="cuda")
    cache[:count] = _filled_cache(case["bits"], count, H, D, g)
    at = torch.arange(n, device="cuda")
    there = at < lens[:, None].clamp(max=n)
    slots = torch.where(there, out_pages.long()[:, at // PAGE] * PAGE + at % PAGE, -1).int()
    return dict(case=case, pages=pages, lens=lens, weights=weights, count=count, out_pages=out_pages, cache=cache,
                max_len=most, slots=slots.flatten(), there=there,
                out_weights=torch.zeros(B, H, n, device="cuda"), kept=torch.zeros(B, H, n, device="cuda", dtype=torch.int32),
                new_lens=torch.zeros(B, device="cuda", dtype=torch.int32),
                k_out=torch.zeros(B * n, H, D, device="cuda", dtype=torch.bfloat16),
                v_out=torch.zeros(B * n, H, D, device="cuda", dtype=torch.bfloat16))


def prepare(case, seed):
    g = _generator(seed)
    s = {"append": _prepare_append, "attend": _prepare_queries, "weights": _prepare_weights,
         "evict": _prepare_evict}[case["op"]](case, g)
    if own:  # what a program keeps beside its tensors: the cache's and the table's descriptions, and workspaces
        import quantized_q8kpack_fp32_amd as q8

        s["q8"] = q8
        if "dtype" in case:
            s["dtype"] = {"f32": q8.Q8K_F32, "f16": q8.Q8K_F16, "bf16": q8.Q8K_BF16}[case["dtype"]]
        pages = s["cache"].shape[0] if case["op"] == "evict" else s["pages"] if case["op"] == "append" else s["count"]
        s["kv"] = q8.KVCache(s["cache"], pages, case["kv_heads"], case["dim"], bits=case.get("bits", 4))
        s["rope"] = None
        if case.get("rot"):
            kind = q8.Q8K_ROPE_HALF if case["pairs"] == "half" else q8.Q8K_ROPE_ADJACENT
            s["rope"] = q8.Rope(s["table"], s["table"].shape[0], case["rot"], kind)
        need = 0
        if case["op"] == "attend":
            need = q8.qattend_kv4_workspace_bytes(s["kv"], case["q_heads"], case["batch"], s["Tq"], s["max_q"],
                                                  s["max_len"])
        if case["op"] == "weights":
            need = q8.qattend_weights_workspace_bytes(s["kv"], case["q_heads"], case["batch"], s["Tq"], s["max_q"],
                                                      s["max_len"])
        s["ws"], s["ws_bytes"] = torch.zeros(max(need, 16), dtype=torch.uint8, device="cuda"), need
    return s


# ---------------------------------------------------------------- append
def _append_plain(s):
    c, D = s["case"], s["case"]["dim"]
    slot = torch.where(s["slots"] >= 0, s["slots"], s["pages"] * PAGE).long()
    page, token = slot // PAGE, slot % PAGE
    k = _rotate(s["k"].float(), s["table"], s["pos"], c["rot"], c["pairs"])
    at = _map(4, D)[token]
    head = torch.arange(c["kv_heads"], device="cuda")[None, :, None]
    s["cache"][page[:, None, None], head, at[:, None]] = _token_bytes(4, k, s["v"].float())
    live = (s["slots"] >= 0)[:, None, None]
    k, v = _held(4, s["cache"][page[:, None, None], head, at[:, None]], D)
    zero = torch.zeros((), device="cuda")
    return torch.where(live, k, zero).bfloat16(), torch.where(live, v, zero).bfloat16()


def _append_own(s):
    q8, n, stride = s["q8"], s["n"], s["row"].stride(0)
    q8.q8k_kv4_append(s["dtype"], s["k"], stride, s["v"], stride, n, s["pos"], s["rope"], s["slots"], s["kv"])
    q8.q8k_kv4_read(q8.Q8K_BF16, s["kv"], s["slots"], n, s["k_out"], s["v_out"])
    return s["k_out"], s["v_out"]


# ---------------------------------------------------------------- attend, weights
def _scores(s):
    """[B, key heads, query heads a key head, max_q, tokens] fp32 scores, -inf where a row does not see the token, and
    the values [B, key heads, tokens, dim]."""
    c = s["case"]
    D, H, G, B, Q = c["dim"], c["kv_heads"], c["q_heads"] // c["kv_heads"], c["batch"], s["max_q"]
    q = _rotate(s["q"].float(), s["table"], s["pos"], c["rot"], c["pairs"]) * s["scale"]
    padded = torch.zeros(B, Q, c["q_heads"], D, device="cuda")
    padded[s["seq_of"], s["index"]] = q
    rows = padded.view(B, Q, H, G, D).permute(0, 2, 3, 1, 4).reshape(B, H, G * Q, D)
    at = torch.full((B, Q), -1, device="cuda", dtype=torch.long)
    at[s["seq_of"], s["index"]] = s["pos"].long()
    # every sequence's pages, one after another: [B, H, L, D]
    L = s["pages"].shape[1] * PAGE
    page = s["pages"].long().clamp(min=0)[:, None, :, None, None]
    raw = s["cache"][page, torch.arange(H, device="cuda")[None, :, None, None, None], _map(s["bits"], D)]
    k, v = _held(s["bits"], raw.flatten(2, 3), D)
    score = torch.matmul(rows, k.transpose(2, 3)).view(B, H, G, Q, L)
    token = torch.arange(L, device="cuda")
    seen = token <= at[:, :, None]
    if c["window"]:
        seen = seen & (token > at[:, :, None] - c["window"])
    return score.masked_fill(~seen[:, None, None], -math.inf), v


def _attend_plain(s):
    c = s["case"]
    D, H, G, B, Q = c["dim"], c["kv_heads"], c["q_heads"] // c["kv_heads"], c["batch"], s["max_q"]
    score, v = _scores(s)
    most = score.amax(-1, keepdim=True)
    p = (score - most).exp()
    total = p.sum(-1, keepdim=True)
    out = torch.matmul((p / total).view(B, H, G * Q, -1), v).view(B, H, G, Q, D).permute(0, 3, 1, 2, 4)
    lse = (most + total.log()).squeeze(-1).permute(0, 3, 1, 2)
    out = out.reshape(B, Q, c["q_heads"], D)[s["seq_of"], s["index"]]
    return out.to(s["q"].dtype), lse.reshape(B, Q, c["q_heads"])[s["seq_of"], s["index"]].contiguous()


def _attend_own(s):
    c, q8 = s["case"], s["q8"]
    q8.qattend_kv4(s["dtype"], s["q"], s["row"].stride(0), c["q_heads"], s["kv"], c["batch"], s["cu_q"], s["Tq"],
                   s["max_q"], s["pages"], s["pages"].shape[1], s["lens"], s["max_len"], s["scale"], c["window"],
                   s["pos"], s["rope"], s["out"], s["lse"], s["ws"], s["ws_bytes"])
    return s["out"], s["lse"]


def _weights_plain(s):
    c = s["case"]
    score, _ = _scores(s)
    lse = torch.full((c["batch"], s["max_q"], c["q_heads"]), math.inf, device="cuda")
    lse[s["seq_of"], s["index"]] = s["lse"]
    lse = lse.view(c["batch"], s["max_q"], c["kv_heads"], -1).permute(0, 2, 3, 1)
    gain = (score - lse[..., None]).exp().sum((2, 3))[..., : s["max_len"]]
    token = torch.arange(s["max_len"], device="cuda")
    first_new = (s["lens"] - s["cu_q"].diff())[:, None, None]
    new = gain
    if s["old"] is not None:
        new = torch.where(token < first_new, s["old"][..., : s["max_len"]] * c["keep"], 0.0) + gain
    there = (token < s["lens"][:, None, None]).expand_as(new)
    s["weights"][..., : s["max_len"]] = torch.where(there, new, s["weights"][..., : s["max_len"]])
    return s["weights"]


def _weights_own(s):
    c, q8 = s["case"], s["q8"]
    q8.qattend_weights(s["dtype"], s["q"], s["row"].stride(0), c["q_heads"], s["kv"], c["batch"], s["cu_q"], s["Tq"],
                       s["max_q"], s["pages"], s["pages"].shape[1], s["lens"], s["max_len"], s["scale"], c["window"],
                       s["pos"], s["rope"], s["lse"], s["old"], c["keep"], s["weights"], s["weights"].stride(1), s["ws"],
                       s["ws_bytes"])
    return s["weights"]


# ---------------------------------------------------------------- evict
def _evict_plain(s):
    c = s["case"]
    B, H, D, n = c["batch"], c["kv_heads"], c["dim"], c["budget"]
    token = torch.arange(s["max_len"], device="cuda")
    lens = s["lens"].long()[:, None, None]
    w = s["weights"][..., : s["max_len"]]
    # whole numbers that order as (held in any case, weight, -place) do; weights are not negative here
    key = (w.view(torch.int32).long() << 31) - token
    key = torch.where((token < c["first"]) | (token >= lens - c["last"]), (1 << 62) - token, key)
    key = torch.where(token < lens, key, -(1 << 62) - token)
    take = min(n, s["max_len"])
    at = key.topk(take, -1).indices
    at = torch.where(at < lens, at, s["max_len"]).sort(-1).values
    at = torch.nn.functional.pad(at, (0, n - take), value=s["max_len"])
    there = at < lens
    s["kept"].copy_(torch.where(there, at, -1))
    safe = torch.where(there, at, 0)
    s["out_weights"].copy_(torch.where(there, w.gather(-1, safe), s["out_weights"]))
    s["new_lens"].copy_(s["lens"].clamp(max=n))
    bytes_of = _map(c["bits"], D)
    head = torch.arange(H, device="cuda")[None, :, None, None]
    to = torch.arange(n, device="cuda")
    page = s["pages"].long()[torch.arange(B, device="cuda")[:, None, None], safe // PAGE].clamp(min=0)
    raw = s["cache"][page[..., None], head, bytes_of[safe % PAGE]]
    page, place = s["out_pages"].long()[:, None, to // PAGE, None], bytes_of[to % PAGE]
    s["cache"][page, head, place] = torch.where(there[..., None], raw, s["cache"][page, head, place])
    k, v = _held(c["bits"], s["cache"][page, head, place].transpose(1, 2), D)
    live = s["there"][..., None, None]
    zero = torch.zeros((), device="cuda")
    return {"kept": s["kept"], "weights": s["out_weights"], "new_lens": s["new_lens"],
            "k": torch.where(live, k, zero).bfloat16().flatten(0, 1), "v": torch.where(live, v, zero).bfloat16().flatten(0, 1)}


def _evict_own(s):
    c, q8 = s["case"], s["q8"]
    q8.q8k_kv_evict(s["kv"], c["batch"], s["pages"], s["pages"].shape[1], s["lens"], s["max_len"], s["weights"],
                    s["weights"].stride(1), c["budget"], c["first"], c["last"], s["out_pages"], s["out_pages"].shape[1],
                    s["out_weights"], s["out_weights"].stride(1), s["kept"], s["new_lens"])
    read = q8.q8k_kv_read if c["bits"] == 8 else q8.q8k_kv4_read
    read(q8.Q8K_BF16, s["kv"], s["slots"], s["slots"].numel(), s["k_out"], s["v_out"])
    return {"kept": s["kept"], "weights": s["out_weights"], "new_lens": s["new_lens"], "k": s["k_out"], "v": s["v_out"]}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"append": _append_own, "attend": _attend_own, "weights": _weights_own, "evict": _evict_own}[op](state)
    return {"append": _append_plain, "attend": _attend_plain, "weights": _weights_plain, "evict": _evict_plain}[op](state)


# ---------------------------------------------------------------- work
def work(case):
    size = 4 if case.get("dtype") == "f32" else 2
    H, D, bits = case["kv_heads"], case["dim"], case.get("bits", 4)
    half = D + 4 if bits == 8 else D // 2 + D // 32 + 4  # bytes of a key or value
    if case["op"] == "append":
        n, row = case["tokens"], H * D
        # keys and values in, the cache's codes and scales out; these in again, bf16 values out
        return {"bytes": n * (2 * row * size + 4 * case["rot"] + 8 + 4 * half * H + 2 * row * 2), "flops": n * row * 8}
    if case["op"] == "evict":
        bytes_ = 0
        for _, length in _lengths(case):
            kept = min(length, case["budget"])
            # weights in; of the kept ones the records in, out and in again, weights, places and bf16 values out
            bytes_ += H * (4 * length + kept * (3 * 2 * half + 8 + 4 * D))
        return {"bytes": bytes_, "flops": bytes_}
    Hq, W = case["q_heads"], case["window"]
    weights = case["op"] == "weights"
    bytes_, flops = 0, 0
    for new, length in _lengths(case):
        first = max(0, length - new - W + 1) if W else 0
        bytes_ += new * Hq * (D * size + 4) + new * 4 * case["rot"]
        if weights:
            bytes_ += (length - first) * H * half + length * H * (8 if case["keep"] else 4)
        else:
            bytes_ += (length - first) * H * 2 * half + new * Hq * D * size
        for i in range(length - new, length):
            flops += (2 if weights else 4) * Hq * D * (min(W, i + 1) if W else i + 1)
    return {"bytes": bytes_, "flops": flops}


# ---------------------------------------------------------------- exact
def _turn64(x, table, pos, rot, pairs):
    """The rotation of pairs as products of complex numbers, in 64 bits."""
    x = x.double()
    if not rot:
        return x
    t = table.double()[pos.long()]
    w = torch.complex(t[:, : rot // 2], t[:, rot // 2:])[:, None]
    if pairs == "half":
        z = torch.complex(x[..., : rot // 2].contiguous(), x[..., rot // 2: rot].contiguous()) * w
        y = torch.cat((z.real, z.imag), -1)
    else:
        z = torch.view_as_complex(x[..., :rot].unflatten(-1, (-1, 2)).contiguous()) * w
        y = torch.view_as_real(z).flatten(-2)
    return torch.cat((y, x[..., rot:]), -1)


def _power64(e):
    """2^e exactly (a library's power need not be)."""
    return (1023 + e.long() << 52).view(torch.float64)


def _values64(bits, raw, dim, which):
    """What a token's bytes stand for, value by value, in 64 bits; which: 0 keys, 1 values."""
    i = torch.arange(dim, device=raw.device)
    if bits == 8:
        code = raw[..., which * dim + i].view(torch.int8).double()
        at = 2 * dim + 4 * which
    else:
        f = raw[..., dim + which * (dim // 32) + i // 32].int()
        e, m = f // 16, f % 16
        factor = torch.where(e > 0, (16 + m) * _power64(e - 19), m * 2.0 ** -18)
        if which == 0:
            w = raw[..., : dim // 2].contiguous().view(torch.int32).long() & 0xffffffff
            j = i % 8
            at = (4 * (j // 2) + 16 * (j % 2) + 2) % 32
            w = w[..., i // 8]
            code = ((w | w << 32) >> at & 15) - 8
        else:
            code = (raw[..., dim // 2 + i // 32 * 16 + i % 16].int() >> (4 * (i // 16 % 2)) & 15) - 8
        code = code.double() * factor
        at = dim + dim // 16 + 4 * which
    return code * raw[..., at: at + 4].contiguous().view(torch.float32).double()


def _each_row(s):
    """(sequence, key head, query head, first row, rows, scores [rows, length] in 64 bits, the head's bytes)."""
    case = s["case"]
    D, G = case["dim"], case["q_heads"] // case["kv_heads"]
    q = _turn64(s["q"], s["table"], s["pos"], case["rot"], case["pairs"])
    first = 0
    for b, (new, length) in enumerate(_lengths(case)):
        row = torch.arange(length - new, length, device="cuda")[:, None]
        token = torch.arange(length, device="cuda")
        hidden = token > row
        if case["window"]:
            hidden |= token <= row - case["window"]
        for h in range(case["kv_heads"]):
            raw = s["cache"][s["pages"][b, : -(-length // PAGE)].long(), h][:, _map(s["bits"], D)].flatten(0, 1)[:length]
            k = _values64(s["bits"], raw, D, 0)
            for a in range(h * G, h * G + G):
                x = (q[first: first + new, a] @ k.T) / math.sqrt(D)
                yield b, h, a, first, new, x.masked_fill(hidden, -math.inf), raw
        first += new


def _lse64(s):
    lse = torch.empty(s["Tq"], s["case"]["q_heads"], dtype=torch.float64, device="cuda")
    for _, _, a, first, new, x, _ in _each_row(s):
        lse[first: first + new, a] = torch.logsumexp(x, -1)
    return lse


def exact(case, seed):
    s = prepare(case, seed)
    D = case["dim"]
    if case["op"] == "append":
        live = (s["slots"] >= 0).double()[:, None, None]

        def held(x):  # the nearest of the 15 evenly spaced values of each group
            x = x.unflatten(-1, (-1, 32))
            top = x.abs().amax(-1, keepdim=True)
            most = top.amax(-2, keepdim=True)
            # 16 steps between powers of two down to 2^-14 of the row's largest, from there on steps of 2^-18; the
            # quotient is one of 32 bits by definition
            r = (top / most).float()
            unit = _power64(((r.view(torch.int32) >> 23) - 127).clamp(min=-14) - 4)
            step = (torch.ceil(r.double() / unit) * unit).clamp(min=2.0 ** -60) * most / 7
            return (torch.round(x / step) * step).flatten(-2) * live

        return held(_turn64(s["k"], s["table"], s["pos"], case["rot"], case["pairs"])), held(s["v"].double())
    if case["op"] == "evict":
        n, H = case["budget"], case["kv_heads"]
        kept = torch.full((case["batch"], H, n), -1, dtype=torch.int32)
        weights = torch.zeros(case["batch"], H, n, dtype=torch.float64)
        k, v = torch.zeros(2, case["batch"], n, H, D, dtype=torch.float64, device="cuda").unbind(0)
        for b, (_, length) in enumerate(_lengths(case)):
            for h in range(H):
                w = s["weights"][b, h, :length].double()
                if length > n:
                    end = length - case["last"]
                    order = torch.sort(w[case["first"]: end], descending=True, stable=True).indices + case["first"]
                    inside = torch.zeros(length, dtype=torch.bool, device="cuda")
                    inside[: case["first"]] = inside[end:] = True
                    inside[order[: n - case["first"] - case["last"]]] = True
                    at = inside.nonzero().flatten()
                else:
                    at = torch.arange(length, device="cuda")
                kept[b, h, : len(at)] = at.int().cpu()
                weights[b, h, : len(at)] = w[at].cpu()
                page = s["pages"][b, at // PAGE].long()
                raw = s["cache"][page[:, None], h, _map(case["bits"], D)[at % PAGE]]
                k[b, : len(at), h] = _values64(case["bits"], raw, D, 0)
                v[b, : len(at), h] = _values64(case["bits"], raw, D, 1)
        new = torch.tensor([min(l, n) for _, l in _lengths(case)], dtype=torch.int32)
        return {"kept": kept, "weights": weights, "new_lens": new, "k": k.flatten(0, 1), "v": v.flatten(0, 1)}
    if case["op"] == "weights":
        got = torch.zeros(case["batch"], case["kv_heads"], s["max_len"] + 5, dtype=torch.float64, device="cuda")
        for b, (new, length) in enumerate(_lengths(case)):
            if s["old"] is not None:
                got[b, :, : length - new] = s["old"][b, :, : length - new].double() * case["keep"]
        for b, h, a, first, new, x, _ in _each_row(s):
            got[b, h, : x.shape[1]] += (x - s["lse"][first: first + new, a, None].double()).exp().sum(0)
        return got
    out = torch.empty(s["Tq"], case["q_heads"], D, dtype=torch.float64, device="cuda")
    lse = torch.empty(s["Tq"], case["q_heads"], dtype=torch.float64, device="cuda")
    v, at = None, None
    for b, h, a, first, new, x, raw in _each_row(s):
        if at != (b, h):
            v, at = _values64(4, raw, D, 1), (b, h)
        total = torch.logsumexp(x, -1)
        lse[first: first + new, a] = total
        out[first: first + new, a] = (x - total[:, None]).exp() @ v
    return out, lse
