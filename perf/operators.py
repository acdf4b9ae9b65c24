"""What is measured of the serving operators that stand around the projections:

  append    new keys are turned by their positions, keys and values are brought to 8 bits and written into a paged
            cache; the values that the cache then holds for these tokens come back (q8k_kv_append, q8k_kv_read)
  attend    softmax attention of new tokens over the paged 8-bit cache, from one token a sequence to whole prompts
            (qattend)
  logprobs  the log probability of a given token in each row of logits, the row's entropy and its top alternatives
            (qlogprobs)

`own` chooses between the library's calls and the plain torch forms.
"""
import math

import torch

own = False

PAGE = 64  # tokens of a cache page
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # one new token of one conversation: the smallest call there is
        dict(name="append_1", op="append", tokens=1, pad=0, kv_heads=8, dim=128, dtype="f32", rot=128, pairs="half"),
        # a decode batch in a padded (graph-captured) step: some of its rows stand for no sequence
        dict(name="append_batch_61", op="append", tokens=61, pad=3, kv_heads=8, dim=128, dtype="f32", rot=128,
             pairs="adjacent"),
        # prompts entering the cache, partial rotation, odd count
        dict(name="append_prompt_8191", op="append", tokens=8191, pad=0, kv_heads=8, dim=128, dtype="bf16", rot=64,
             pairs="half"),
        # one conversation's next token after a short prompt
        dict(name="decode_1x513", op="attend", batch=1, q=1, len=513, ragged=False, q_heads=32, kv_heads=8, dim=128,
             dtype="f32", window=0, rot=128, pairs="half"),
        # a decode batch of conversations of many lengths
        dict(name="decode_16x8191", op="attend", batch=16, q=1, len=8191, ragged=True, q_heads=32, kv_heads=8, dim=128,
             dtype="f32", window=0, rot=128, pairs="adjacent"),
        # decode over long documents
        dict(name="decode_8x65537", op="attend", batch=8, q=1, len=65537, ragged=False, q_heads=32, kv_heads=8,
             dim=128, dtype="bf16", window=0, rot=0, pairs="half"),
        # several drafted tokens a sequence checked at once, every head with its own keys, a sliding window
        dict(name="verify_12x5_w1000", op="attend", batch=12, q=5, len=2900, ragged=True, q_heads=16, kv_heads=16,
             dim=64, dtype="f16", window=1000, rot=32, pairs="half"),
        # a prompt of 512 tokens from its start
        dict(name="prompt_512", op="attend", batch=1, q=512, len=512, ragged=False, q_heads=32, kv_heads=8, dim=128,
             dtype="f32", window=0, rot=128, pairs="half"),
        # chunks of long prompts, over what of them the cache already holds
        dict(name="chunk_3x1000_16001", op="attend", batch=3, q=1000, len=16001, ragged=True, q_heads=32, kv_heads=4,
             dim=128, dtype="bf16", window=0, rot=128, pairs="half"),
        # the token just chosen, with the usual handful of alternatives
        dict(name="logprobs_1x32000", op="logprobs", rows=1, vocab=32000, dtype="f32", top=5),
        # a decode batch over a large odd vocabulary
        dict(name="logprobs_48x128257", op="logprobs", rows=48, vocab=128257, dtype="bf16", top=20),
        # scoring a prompt of 512 tokens
        dict(name="logprobs_512x32000", op="logprobs", rows=512, vocab=32000, dtype="f32", top=8),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "attend", "logprobs"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    dim = rng.choice([64, 128, 128, 256])
    rot = rng.choice([0, dim, dim, dim // 2])
    pairs = rng.choice(["half", "adjacent"])
    if op == "append":
        kv_heads = rng.choice([1, 2, 4, 8, 16])
        tokens = _log(rng, 1, min(8191, 8191 * 1024 // (kv_heads * dim)))
        return dict(op=op, tokens=tokens, pad=rng.choice([0, 0, 1, 7]), kv_heads=kv_heads, dim=dim, dtype=dtype,
                    rot=rot, pairs=pairs)
    if op == "logprobs":
        vocab = _log(rng, 1000, 160000)
        return dict(op=op, rows=_log(rng, 1, max(1, 512 * 32000 // vocab)), vocab=vocab, dtype=dtype,
                    top=rng.choice([0, 1, 5, 20, 32]))
    kv_heads = rng.choice([1, 2, 4, 8])
    q_heads = kv_heads * rng.choice([1, 2, 4, 6, 8])
    if rng.random() < 0.6:  # decode, or a few drafted tokens
        q = rng.choice([1, 1, 1, 2, 5, 8])
        batch = _log(rng, 1, 64)
        top = (8 * 65537 * 8 * 128) // (batch * kv_heads * dim)
        length = _log(rng, max(q, 16), max(64, min(65537, top)))
    else:  # prompts and chunks of them
        q = _log(rng, 16, 1000)
        batch = rng.choice([1, 1, 2, 3, 5])
        # cost (and the plain form's score matrix) at most about half of chunk_3x1000_16001's
        top = (500 * 16001 * 32 * 3) // (batch * q * q_heads * max(1, dim // 128))
        length = _log(rng, q, max(q, min(16001, top)))
    return dict(op="attend", batch=batch, q=q, len=length, ragged=rng.random() < 0.7, q_heads=q_heads,
                kv_heads=kv_heads, dim=dim, dtype=dtype, window=rng.choice([0, 0, 0, max(1, length // 3)]), rot=rot,
                pairs=pairs)


def _lengths(case):
    """(new tokens, cached tokens with the new ones) of each sequence: the first has the most of both, the others
    spread evenly below that where the case is ragged."""
    got = []
    for b in range(case["batch"]):
        f = (b * 0.6180339887498949) % 1.0 if case["ragged"] else 0.0
        new = max(1, int(case["q"] * (1.0 - 0.9 * f)))
        got.append((new, max(new, int(case["len"] * (1.0 - 0.9 * f)))))
    return got


# ---------------------------------------------------------------- the cache
# One record for each page and key head: keys in planes of 64 of the head's values [dim/64][64 tokens][64], values
# turned round [dim][64 places], one fp32 scale for each token's keys [64] and values [64].  Token t of a page has
# the place (t>>2 & 3) << 4 | (t>>5) << 3 | (t>>4 & 1) << 2 | (t & 3) in a row of values.


def _record_bytes(dim):
    return 2 * PAGE * dim + 8 * PAGE


def _places(t):
    return ((t >> 2) & 3) << 4 | (t >> 5) << 3 | ((t >> 4) & 1) << 2 | (t & 3)


def _parts(cache, dim):
    """Views of a cache's codes and scales: [page, head, plane, token, 64], [page, head, dim, place], 2 x [page, head, token]."""
    k = cache[..., : PAGE * dim].unflatten(-1, (dim // 64, PAGE, 64))
    v = cache[..., PAGE * dim: 2 * PAGE * dim].unflatten(-1, (dim, PAGE))
    s = cache.view(torch.float32)[..., PAGE * dim // 2:]
    return k, v, s[..., :PAGE], s[..., PAGE:]


def _quantise(x):
    """Codes (as float) and scale of the last axis: the scale is the largest magnitude / 127."""
    most = x.abs().amax(-1, keepdim=True)
    codes = torch.where(most > 0, torch.round(x * (127.0 / most)).clamp(-127, 127), torch.zeros_like(x))
    return codes, (most / 127.0).squeeze(-1)


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
    row = row.to(dt)
    # pages handed out in no order; tokens run on from the middle of the first page
    count = (T + 37 + PAGE - 1) // PAGE + 5
    order = torch.randperm(count, device="cuda", generator=g)
    at = torch.arange(T, device="cuda") + 37
    slots = torch.cat([order[at // PAGE] * PAGE + at % PAGE, torch.full((case["pad"],), -1, device="cuda")]).int()
    pos = torch.cat([at, torch.zeros(case["pad"], device="cuda", dtype=at.dtype)]).int()
    table = _rope_table(T + 37, case["rot"]) if case["rot"] else None
    # one page more than the cache has: the plain form's place for rows that stand for no token
    cache = torch.zeros(count + 1, H, _record_bytes(D), dtype=torch.int8, device="cuda")
    s = dict(case=case, row=row, k=row[:, 4 * H: 5 * H], v=row[:, 5 * H:], slots=slots, pos=pos, table=table,
             cache=cache, pages=count, n=n, k_out=torch.zeros(n, H, D, device="cuda", dtype=torch.bfloat16),
             v_out=torch.zeros(n, H, D, device="cuda", dtype=torch.bfloat16))
    return s


def _prepare_attend(case, g):
    B, Hq, H, D = case["batch"], case["q_heads"], case["kv_heads"], case["dim"]
    seqs = _lengths(case)
    per = [(l + PAGE - 1) // PAGE for _, l in seqs]
    count, most = sum(per), max(per)
    cache = torch.empty(count, H, _record_bytes(D), dtype=torch.int8, device="cuda")
    kc, vc, ks, vs = _parts(cache, D)
    # keys whose products with the queries spread as trained heads' do: a few channels stand out
    lift = torch.rand(H, D, device="cuda", generator=g) ** 4 * 2 + 0.5
    place = torch.empty(PAGE, dtype=torch.long, device="cuda")
    place[_places(torch.arange(PAGE, device="cuda"))] = torch.arange(PAGE, device="cuda")
    for p in range(0, count, 256):
        m = min(count, p + 256) - p
        c, sc = _quantise(torch.randn(m, H, PAGE, D, device="cuda", generator=g) * lift[:, None])
        kc[p: p + m] = c.to(torch.int8).unflatten(-1, (D // 64, 64)).transpose(2, 3)
        ks[p: p + m] = sc
        c, sc = _quantise(torch.randn(m, H, PAGE, D, device="cuda", generator=g))
        vc[p: p + m] = c.to(torch.int8).transpose(2, 3)[..., place]
        vs[p: p + m] = sc
    order = torch.randperm(count, device="cuda", generator=g).int()
    pages = torch.full((B, most), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(per):
        pages[b, :n] = order[at: at + n]
        at += n
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
    s = dict(case=case, q=row[:, :Hq], row=row, cache=cache, pages=pages, lens=lens, cu_q=cu_q, pos=pos, Tq=Tq,
             seq_of=seq_of, index=index, max_q=max(n for n, _ in seqs), max_len=max(l for _, l in seqs), count=count,
             table=_rope_table(case["len"], case["rot"]) if case["rot"] else None, scale=1.0 / math.sqrt(D),
             out=torch.zeros(Tq, Hq, D, device="cuda", dtype=row.dtype), lse=torch.zeros(Tq, Hq, device="cuda"))
    return s


def _prepare_logprobs(case, g):
    T, V, n = case["rows"], case["vocab"], case["top"]
    x = torch.randn(T, V, device="cuda", generator=g) * 2.5
    # a few tokens stand out in each row, as after training; the last tokens of the vocabulary are banned
    at = torch.randint(0, V, (T, 12), device="cuda", generator=g)
    x.scatter_(1, at, torch.rand(T, 12, device="cuda", generator=g) * 14 + 4)
    x[:, V - V // 500:] = -math.inf
    targets = torch.where(torch.rand(T, device="cuda", generator=g) < 0.7, at[:, 0],
                          torch.randint(0, V, (T,), device="cuda", generator=g)).int()
    f = dict(device="cuda", dtype=torch.float32)
    return dict(case=case, logits=x.to(TYPES[case["dtype"]]), targets=targets, logprob=torch.zeros(T, **f),
                entropy=torch.zeros(T, **f), lse=torch.zeros(T, **f),
                top_ids=torch.zeros(T, n, device="cuda", dtype=torch.int32), top_logprob=torch.zeros(T, n, **f))


def prepare(case, seed):
    g = _generator(seed)
    s = {"append": _prepare_append, "attend": _prepare_attend, "logprobs": _prepare_logprobs}[case["op"]](case, g)
    if own:  # what a program keeps beside its tensors: the cache's and the table's descriptions, and workspaces
        import quantized_q8kpack_fp32_amd as q8

        s["q8"] = q8
        s["dtype"] = {"f32": q8.Q8K_F32, "f16": q8.Q8K_F16, "bf16": q8.Q8K_BF16}[case["dtype"]]
        need = 0
        if case["op"] != "logprobs":
            s["kv"] = q8.KVCache(s["cache"], s["pages"] if case["op"] == "append" else s["count"], case["kv_heads"],
                                 case["dim"])
            s["rope"] = None
            if case["rot"]:
                kind = q8.Q8K_ROPE_HALF if case["pairs"] == "half" else q8.Q8K_ROPE_ADJACENT
                s["rope"] = q8.Rope(s["table"], s["table"].shape[0], case["rot"], kind)
        if case["op"] == "attend":
            need = q8.qattend_workspace_bytes(s["kv"], case["q_heads"], case["batch"], s["Tq"], s["max_q"],
                                              s["max_len"])
        if case["op"] == "logprobs":
            need = q8.qlogprobs_workspace_bytes(case["rows"], case["vocab"], case["top"])
        s["ws"], s["ws_bytes"] = torch.zeros(max(need, 16), dtype=torch.uint8, device="cuda"), need
    return s


# ---------------------------------------------------------------- append
def _append_plain(s):
    c, D = s["case"], s["case"]["dim"]
    kc, vc, ks, vs = _parts(s["cache"], D)
    slot = torch.where(s["slots"] >= 0, s["slots"], s["pages"] * PAGE).long()
    page, token = slot // PAGE, slot % PAGE
    k, kscale = _quantise(_rotate(s["k"].float(), s["table"], s["pos"], c["rot"], c["pairs"]))
    v, vscale = _quantise(s["v"].float())
    kc[page, :, :, token] = k.to(torch.int8).unflatten(-1, (D // 64, 64))
    vc[page, :, :, _places(token)] = v.to(torch.int8)
    ks[page, :, token] = kscale
    vs[page, :, token] = vscale
    live = (s["slots"] >= 0)[:, None, None]
    k = kc[page, :, :, token].flatten(2).float() * ks[page, :, token][..., None]
    v = vc[page, :, :, _places(token)].float() * vs[page, :, token][..., None]
    zero = torch.zeros((), device="cuda")
    return torch.where(live, k, zero).bfloat16(), torch.where(live, v, zero).bfloat16()


def _append_own(s):
    q8, n, stride = s["q8"], s["n"], s["row"].stride(0)
    q8.q8k_kv_append(s["dtype"], s["k"], stride, s["v"], stride, n, s["pos"], s["rope"], s["slots"], s["kv"])
    q8.q8k_kv_read(q8.Q8K_BF16, s["kv"], s["slots"], n, s["k_out"], s["v_out"])
    return s["k_out"], s["v_out"]


# ---------------------------------------------------------------- attend
def _attend_plain(s):
    c = s["case"]
    D, H, G, B, Q = c["dim"], c["kv_heads"], c["q_heads"] // c["kv_heads"], c["batch"], s["max_q"]
    q = _rotate(s["q"].float(), s["table"], s["pos"], c["rot"], c["pairs"]) * s["scale"]
    padded = torch.zeros(B, Q, c["q_heads"], D, device="cuda")
    padded[s["seq_of"], s["index"]] = q
    rows = padded.view(B, Q, H, G, D).permute(0, 2, 3, 1, 4).reshape(B, H, G * Q, D)
    at = torch.zeros(B, Q, device="cuda", dtype=torch.long)
    at[s["seq_of"], s["index"]] = s["pos"].long()
    # every sequence's pages, one after another: [B, H, L, D]
    kc, vc, ks, vs = _parts(s["cache"], D)
    page = s["pages"].long().clamp(min=0)
    L = page.shape[1] * PAGE
    k = (kc[page].float() * ks[page][:, :, :, None, :, None]).permute(0, 2, 1, 4, 3, 5).reshape(B, H, L, D)
    order = _places(torch.arange(PAGE, device="cuda"))
    v = (vc[page][..., order].float() * vs[page][:, :, :, None, :]).permute(0, 2, 1, 4, 3).reshape(B, H, L, D)
    score = torch.matmul(rows, k.transpose(2, 3)).view(B, H, G, Q, L)
    token = torch.arange(L, device="cuda")
    seen = token <= at[:, :, None]
    if c["window"]:
        seen = seen & (token > at[:, :, None] - c["window"])
    score = score.masked_fill(~seen[:, None, None], -math.inf)
    most = score.amax(-1, keepdim=True)
    p = (score - most).exp()
    total = p.sum(-1, keepdim=True)
    out = torch.matmul((p / total).view(B, H, G * Q, L), v).view(B, H, G, Q, D).permute(0, 3, 1, 2, 4)
    lse = (most + total.log()).squeeze(-1).permute(0, 3, 1, 2)
    out = out.reshape(B, Q, c["q_heads"], D)[s["seq_of"], s["index"]]
    return out.to(s["q"].dtype), lse.reshape(B, Q, c["q_heads"])[s["seq_of"], s["index"]].contiguous()


def _attend_own(s):
    c, q8 = s["case"], s["q8"]
    q8.qattend(s["dtype"], s["q"], s["row"].stride(0), c["q_heads"], s["kv"], c["batch"], s["cu_q"], s["Tq"],
               s["max_q"], s["pages"], s["pages"].shape[1], s["lens"], s["max_len"], s["scale"], c["window"],
               s["pos"], s["rope"], s["out"], s["lse"], s["ws"], s["ws_bytes"])
    return s["out"], s["lse"]


# ---------------------------------------------------------------- logprobs
def _logprobs_plain(s):
    c = s["case"]
    x = s["logits"].float()
    m = x.amax(-1, keepdim=True)
    d = x - m
    e = d.exp()
    z = e.sum(-1, keepdim=True)
    lse = m + z.log()
    entropy = z.log() - torch.where(e > 0, e * d, torch.zeros_like(e)).sum(-1, keepdim=True) / z
    logprob = x.gather(1, s["targets"].long()[:, None]) - lse
    # the largest first, equal ones by their place: whole numbers that order as (logit, -place) do
    bits = (x + 0.0).view(torch.int32).long()
    key = torch.where(bits < 0, -(bits & 0x7fffffff), bits) * (1 << 32) - torch.arange(c["vocab"], device="cuda")
    ids = key.topk(c["top"], -1).indices if c["top"] else torch.zeros(c["rows"], 0, device="cuda", dtype=torch.long)
    return {"logprob": logprob.squeeze(1), "entropy": entropy.squeeze(1), "lse": lse.squeeze(1),
            "top_ids": ids.int(), "top_logprob": x.gather(1, ids) - lse}


def _logprobs_own(s):
    c, q8 = s["case"], s["q8"]
    q8.qlogprobs(s["dtype"], s["logits"], s["logits"].stride(0), c["rows"], c["vocab"], s["targets"], s["logprob"],
                 s["entropy"], s["lse"], c["top"], s["top_ids"], s["top_logprob"], s["ws"], s["ws_bytes"])
    return {k: s[k] for k in ("logprob", "entropy", "lse", "top_ids", "top_logprob")}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"append": _append_own, "attend": _attend_own, "logprobs": _logprobs_own}[op](state)
    return {"append": _append_plain, "attend": _attend_plain, "logprobs": _logprobs_plain}[op](state)


# ---------------------------------------------------------------- work
def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "append":
        n, row = case["tokens"], case["kv_heads"] * case["dim"]
        held = 2 * row + 8 * case["kv_heads"]
        # keys and values in, the cache's codes and scales out; these in again, bf16 values out
        return {"bytes": n * (2 * row * size + 4 * case["rot"] + 8 + 2 * held + 2 * row * 2),
                "flops": n * row * 8}
    if case["op"] == "logprobs":
        T, V, n = case["rows"], case["vocab"], case["top"]
        return {"bytes": T * (V * size + 4 + 12 + 8 * n), "flops": 6 * T * V}
    Hq, H, D, W = case["q_heads"], case["kv_heads"], case["dim"], case["window"]
    bytes_, flops = 0, 0
    for new, length in _lengths(case):
        first = max(0, length - new - W + 1) if W else 0
        bytes_ += (length - first) * H * (2 * D + 8) + new * Hq * (2 * D * size + 4) + new * 4 * case["rot"]
        for i in range(length - new, length):
            flops += 4 * Hq * D * (min(W, i + 1) if W else i + 1)
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


def exact(case, seed):
    s = prepare(case, seed)
    D = case["dim"] if case["op"] != "logprobs" else 0
    if case["op"] == "append":
        live = (s["slots"] >= 0).double()[:, None, None]

        def held(x):  # the nearest of the 255 evenly spaced values that reach the largest magnitude
            step = x.abs().amax(-1, keepdim=True) / 127
            return torch.round(x / step) * step * live

        return held(_turn64(s["k"], s["table"], s["pos"], case["rot"], case["pairs"])), held(s["v"].double())
    if case["op"] == "logprobs":
        x = s["logits"].double()
        lse = torch.logsumexp(x, -1)
        p = (x - lse[:, None]).exp()
        entropy = -(p * (x - lse[:, None]).clamp(min=-1e300)).sum(-1)
        order = torch.sort(x, dim=-1, descending=True, stable=True)
        n = case["top"]
        return {"logprob": x[torch.arange(len(x)), s["targets"].long()] - lse, "entropy": entropy, "lse": lse,
                "top_ids": order.indices[:, :n].int(), "top_logprob": order.values[:, :n] - lse[:, None]}
    G = case["q_heads"] // case["kv_heads"]
    q = _turn64(s["q"], s["table"], s["pos"], case["rot"], case["pairs"])
    out = torch.empty(s["Tq"], case["q_heads"], D, dtype=torch.float64, device="cuda")
    lse = torch.empty(s["Tq"], case["q_heads"], dtype=torch.float64, device="cuda")
    at = torch.tensor([(t >> 2 & 3) * 16 + (t >> 5) * 8 + (t >> 4 & 1) * 4 + t % 4 for t in range(PAGE)], device="cuda")
    first = 0
    for b, (new, length) in enumerate(_lengths(case)):
        mine = s["cache"][s["pages"][b, : -(-length // PAGE)].long()]
        row = torch.arange(length - new, length, device="cuda")[:, None]
        token = torch.arange(length, device="cuda")
        hidden = token > row
        if case["window"]:
            hidden |= token <= row - case["window"]
        for h in range(case["kv_heads"]):
            rec = mine[:, h].contiguous()
            scale = rec[:, 2 * PAGE * D:].view(torch.float32).double()
            k = rec[:, : PAGE * D].reshape(-1, D // 64, PAGE, 64).transpose(1, 2).reshape(-1, D).double()
            v = rec[:, PAGE * D: 2 * PAGE * D].reshape(-1, D, PAGE)[:, :, at].transpose(1, 2).reshape(-1, D).double()
            k = (k * scale[:, :PAGE].reshape(-1, 1))[:length]
            v = (v * scale[:, PAGE:].reshape(-1, 1))[:length]
            for g in range(h * G, h * G + G):
                x = (q[first: first + new, g] @ k.T) / math.sqrt(D)
                x = x.masked_fill(hidden, -math.inf)
                total = torch.logsumexp(x, -1)
                lse[first: first + new, g] = total
                out[first: first + new, g] = (x - total[:, None]).exp() @ v
        first += new
    return out, lse
