"""The operators between the projections on the GPU, against plain numpy forms
(serving_helpers.py): the paged 8-bit cache byte for byte, attention and log
probabilities within bounds derived there."""
import numpy as np
import pytest

import serving_helpers as sh
from gpu_helpers import host, poisoned, to_dev
from serving_helpers import assert_exact, assert_within, back, q_dtype, record, round_to, to_dev_as, torch_dtype, tracked

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import quantized_q8kpack_fp32_amd as q

    return tracked(q)


def rope_of(q, table, pairs):
    if table is None:
        return None
    return q.Rope(to_dev(table), table.shape[0], table.shape[1],
                  q.Q8K_ROPE_HALF if pairs == "half" else q.Q8K_ROPE_ADJACENT)


def cache_of(q, host_cache, D):
    """A device cache holding `host_cache`, uint8 [pages][heads][record(D)]."""
    return q.KVCache(to_dev(host_cache), host_cache.shape[0], host_cache.shape[1], D)


def poisoned_cache(pages, heads, D):
    return np.full((pages, heads, record(D)), 0xFF, np.uint8)


def cache_bytes(kv, pages, heads, D):
    return host(kv.data)[: pages * heads * record(D)].reshape(pages, heads, record(D))


# ---------------------------------------------------------------------- append
APPEND = [
    # D, dtype, pairs, rot, heads, tokens
    (64, "f32", "half", 64, 1, 1),
    (128, "f32", "half", 128, 8, 1),
    (256, "f32", "half", 256, 2, 3),
    (128, "f32", "adjacent", 128, 8, 61),
    (128, "bf16", "half", 64, 3, 130),
    (64, "f16", "adjacent", 32, 5, 77),
    (256, "bf16", "adjacent", 8, 1, 65),
    (256, "f16", "half", 128, 4, 200),
    (64, "f32", "half", 0, 2, 129),
    (128, "f16", "half", 8, 1, 700),
    # tokens by the tile
    (64, "bf16", "adjacent", 64, 16, 521),
    (256, "f32", "half", 128, 32, 257),
    (128, "f16", "half", 128, 8, 1030),
]


def append_case(D, dtype, heads, T, seed, scattered=True):
    g = np.random.default_rng(seed)
    row = round_to(g.standard_normal((T, 3 * heads, D)) * g.uniform(0.01, 8, (T, 3 * heads, 1)), dtype)
    if T > 4:
        row[1, heads:] = 0  # a head of nothing but zeros
        row[2, heads:] = round_to(np.full((2 * heads, D), 1e-42), dtype)  # 127/amax overflows
        row[3, heads:, 5] = round_to(np.float32(3e4), dtype)  # one large value
    pages = max(4, 2 * (T // 64 + 2))
    slots = g.permutation(pages * 64)[:T].astype(np.int32) if scattered else (37 + np.arange(T)).astype(np.int32)
    if T > 8:
        slots[5], slots[6], slots[7] = -1, pages * 64, 2 ** 31 - 1
    return g, row, pages, slots


@pytest.mark.parametrize("D,dtype,pairs,rot,heads,T", APPEND)
@pytest.mark.parametrize("scattered", [True, False])
def test_append(q, D, dtype, pairs, rot, heads, T, scattered):
    g, row, pages, slots = append_case(D, dtype, heads, T, 11 + T, scattered)
    if not scattered and T > 200:  # and runs with breaks, of every length and start
        slots[100:] += 5
        slots[150:] += 64
        slots[170:180] = slots[170:180][::-1].copy()
    table = sh.rope_table(g, 300, rot) if rot else None
    pos = g.integers(0, 300, T).astype(np.int32)
    if T > 16 and rot:
        pos[9], pos[10] = 300, -1  # outside the table: not written
    want = poisoned_cache(pages, heads, D)
    sh.append(want, row[:, heads: 2 * heads], row[:, 2 * heads:], table, pos, pairs, slots, D)
    kv = cache_of(q, poisoned_cache(pages, heads, D), D)
    rd = to_dev_as(row, dtype)
    q.q8k_kv_append(q_dtype(q, dtype), rd[:, heads: 2 * heads], 3 * heads * D, rd[:, 2 * heads:], 3 * heads * D, T,
                    to_dev(pos), rope_of(q, table, pairs), to_dev(slots), kv)
    assert_exact(cache_bytes(kv, pages, heads, D), want, f"cache {D} {dtype} {pairs} {rot}")


def test_append_one_by_one_and_at_once(q):
    """Appends touch no token but their own: any cutting into calls gives the same bytes."""
    D, heads, T = 128, 16, 520
    g, row, pages, slots = append_case(D, "f32", heads, T, 5, scattered=False)
    table = sh.rope_table(g, T, D)
    pos = np.arange(T, dtype=np.int32)
    rd, pd, sd = to_dev_as(row, "f32"), to_dev(pos), to_dev(slots)
    rope = rope_of(q, table, "half")

    def run(cuts):
        kv = cache_of(q, poisoned_cache(pages, heads, D), D)
        for a, b in zip(cuts, cuts[1:]):
            q.q8k_kv_append(q.Q8K_F32, rd[a:b, heads: 2 * heads], 3 * heads * D, rd[a:b, 2 * heads:], 3 * heads * D,
                            b - a, pd[a:b], rope, sd[a:b], kv)
        return cache_bytes(kv, pages, heads, D)

    want = poisoned_cache(pages, heads, D)
    sh.append(want, row[:, heads: 2 * heads], row[:, 2 * heads:], table, pos, "half", slots, D)
    for cuts in ([0, T], list(range(T + 1)), [0, 1, 3, T]):
        assert_exact(run(cuts), want, f"cuts {cuts[:4]}")


@pytest.mark.parametrize("D,heads,T", [(64, 1, 1), (128, 8, 70), (256, 3, 333), (64, 4, 1000), (64, 16, 600), (256, 32, 259), (128, 9, 1000)])
@pytest.mark.parametrize("dtype", sh.DTYPES)
def test_read(q, D, heads, T, dtype):
    g = np.random.default_rng(T)
    pages = 20
    raw = g.integers(0, 256, (pages, heads, record(D)), dtype=np.uint8)
    raw[..., 2 * 64 * D:] = np.abs(g.standard_normal((pages, heads, 128))).astype(np.float32).view(np.uint8)
    slots = g.integers(0, pages * 64, T).astype(np.int32)  # repeats are fine
    if T > 3:
        slots[0], slots[1], slots[2] = -5, pages * 64, 2 ** 31 - 1
        slots[T // 2:] = 64 + np.arange(T - T // 2)
    k, ks, v, vs = sh.held(raw, slots, D)
    import torch

    kd = torch.full((T, heads, D), float("nan"), dtype=torch_dtype(dtype), device="cuda")
    vd = kd.clone()
    q.q8k_kv_read(q_dtype(q, dtype), cache_of(q, raw, D), to_dev(slots), T, kd, vd)
    assert_exact(back(kd), round_to(k.astype(np.float32) * ks[..., None], dtype), "keys")
    assert_exact(back(vd), round_to(v.astype(np.float32) * vs[..., None], dtype), "values")


# ---------------------------------------------------------------------- attend
def attend_case(D, heads, lens, news, seed, spare=3, spread=1.0):
    """A cache of random codes whose places beyond the sequences hold NaN scales,
    its page table (places beyond a sequence's pages point outside the cache)."""
    g = np.random.default_rng(seed)
    per = [-(-n // 64) for n in lens]
    pages = sum(per) + spare
    raw = g.integers(0, 256, (pages, heads, record(D)), dtype=np.uint8)
    codes = raw[..., : 128 * D].view(np.int8)
    codes[codes == -128] = -127
    sc = raw[..., 128 * D:].view(np.float32)
    sc[:] = np.nan
    order = g.permutation(pages).astype(np.int32)
    most = max(per + [1])
    table = np.full((len(lens), most), -1, np.int32)
    table[:, 1::2] = 2 ** 30
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = order[at: at + n]
        at += n
        for i in range(lens[b]):
            r = sc[table[b, i // 64]]
            r[:, i % 64] = g.uniform(0.2, 2.0, heads) / 73 * spread
            r[:, 64 + i % 64] = 10.0 ** g.uniform(-3, 1, heads) / 73
    cu = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
    return g, raw, table, cu


def run_attend(q, raw, table, cu, lens, qx, D, dtype, window, rope_table, pos, pairs, extra_rows=2, max_len=None,
               max_q=None, scale=None, lse=True):
    import torch

    Tq, Hq = qx.shape[0], qx.shape[1]
    kv = cache_of(q, raw, D)
    qd = torch.full((Tq + extra_rows, Hq + 3, D), float("nan"), dtype=torch_dtype(dtype), device="cuda")
    qd[:Tq, :Hq] = to_dev_as(qx, dtype)
    out = torch.full((Tq + extra_rows, Hq, D), 7.0, dtype=torch_dtype(dtype), device="cuda")
    ls = torch.full((Tq + extra_rows, Hq), 7.0, device="cuda")
    max_len = int(max(lens)) if max_len is None else max_len
    max_q = int(np.diff(cu).max()) if max_q is None else max_q
    B = len(lens)
    need = q.qattend_workspace_bytes(kv, Hq, B, Tq + extra_rows, max_q, max_len)
    ws = poisoned(need) if need else None
    pd = to_dev(np.concatenate([pos, np.full(extra_rows, -1, np.int32)])) if pos is not None else None
    q.qattend(q_dtype(q, dtype), qd, (Hq + 3) * D, Hq, kv, B, to_dev(cu), Tq + extra_rows, max_q, to_dev(table),
              table.shape[1], to_dev(np.asarray(lens, np.int32)), max_len, D ** -0.5 if scale is None else scale, window,
              pd, rope_of(q, rope_table, pairs), out, ls if lse else None, ws, need)
    o, l = back(out), back(ls)
    assert (o[Tq:] == 7.0).all() and (l[Tq:] == 7.0).all(), "rows of no sequence were written"
    return o[:Tq], l[:Tq]


ATTEND = [
    # D, dtype, q_heads, heads, lens, new tokens, window, rot, pairs
    (128, "f32", 4, 1, [1], [1], 0, 128, "half"),
    (128, "f32", 32, 8, [65], [1], 0, 128, "half"),
    (64, "f32", 1, 1, [63, 64, 65, 1, 0, 128], [1, 1, 1, 1, 1, 1], 0, 64, "adjacent"),
    (128, "f32", 8, 2, [513, 0, 200, 3], [1, 0, 1, 1], 0, 128, "adjacent"),
    (256, "f32", 6, 2, [300, 17], [1, 3], 0, 256, "half"),
    (128, "bf16", 8, 1, [700, 64], [2, 1], 0, 64, "half"),
    (64, "f16", 16, 16, [190, 64, 5], [5, 4, 5], 100, 32, "half"),
    (128, "f32", 12, 4, [333, 129], [7, 1], 1, 0, "half"),
    (64, "bf16", 7, 1, [90], [3], 63, 8, "adjacent"),
    (256, "f16", 2, 2, [130, 20], [20, 20], 64, 128, "adjacent"),
    (256, "bf16", 24, 1, [257], [1], 0, 0, "half"),
    (256, "bf16", 2, 1, [66, 70], [1, 2], 0, 256, "half"),
    (128, "bf16", 10, 5, [129], [1], 0, 0, "half"),
    # more new tokens than length: the first see nothing
    (128, "f32", 4, 2, [3, 2], [5, 2], 0, 0, "half"),
    # long enough for splits; a window that leaves most of them out
    (128, "f32", 4, 1, [5000, 777], [1, 2], 0, 128, "half"),
    (64, "f32", 8, 2, [9000], [2], 500, 64, "half"),
    (64, "bf16", 2, 1, [4097], [1], 4000, 0, "half"),
    (256, "f32", 2, 1, [3333], [1], 0, 0, "half"),
    # prompts and chunks
    (128, "f32", 8, 2, [200, 333], [200, 70], 0, 128, "half"),
    (128, "bf16", 4, 4, [257, 64], [130, 64], 0, 128, "adjacent"),
    (64, "f16", 8, 1, [150], [150], 40, 64, "half"),
    (256, "f32", 4, 2, [190, 1], [150, 1], 0, 256, "half"),
    (64, "f32", 4, 2, [1100, 900], [40, 33], 0, 0, "half"),
    (256, "bf16", 2, 1, [300], [300], 0, 0, "half"),
    (128, "f16", 6, 2, [400, 410, 1], [90, 100, 1], 130, 64, "half"),
    (64, "bf16", 6, 2, [190], [60], 0, 64, "half"),
    (64, "bf16", 6, 2, [190], [60], 33, 0, "half"),
    (256, "bf16", 3, 1, [100, 50], [31, 50], 0, 128, "half"),
    (128, "bf16", 3, 1, [100, 50], [31, 50], 0, 0, "half"),
    # few tiles of a long sequence
    (64, "bf16", 8, 2, [1000, 800], [33, 12], 0, 64, "half"),
    (64, "bf16", 8, 2, [1000, 800], [33, 12], 0, 0, "half"),
    (64, "f16", 8, 2, [1000, 800], [33, 12], 700, 32, "half"),
    (128, "f32", 8, 2, [1000, 800, 0], [33, 12, 0], 0, 128, "adjacent"),
    (128, "bf16", 8, 2, [1000, 800], [33, 12], 900, 64, "half"),
    (128, "bf16", 8, 2, [1000, 800], [33, 12], 0, 0, "half"),
    (256, "f32", 4, 1, [1000], [33], 0, 256, "half"),
    (256, "bf16", 4, 1, [1000], [33], 0, 64, "half"),
    # whole ones of an odd and an even number of pages
    (128, "f32", 16, 16, [450, 449, 65, 1], [40, 65, 65, 1], 0, 128, "half"),
    (64, "bf16", 16, 16, [450, 449, 385], [40, 65, 65], 200, 0, "half"),
    (128, "f32", 32, 16, [4200], [40], 4100, 128, "half"),
    (128, "bf16", 64, 64, [2048, 300], [100, 90], 0, 128, "half"),
    # many heads: enough of the larger tiles
    (64, "f32", 128, 128, [129, 140], [129, 70], 0, 64, "half"),
    (64, "bf16", 128, 128, [150, 3], [140, 3], 0, 32, "adjacent"),
    (64, "bf16", 128, 128, [150], [150], 0, 0, "half"),
    (128, "f32", 128, 128, [200, 140], [129, 70], 50, 128, "half"),
    (128, "bf16", 128, 128, [150, 3], [140, 3], 0, 32, "adjacent"),
    (128, "bf16", 128, 128, [150], [150], 0, 0, "half"),
    (256, "f16", 128, 128, [129, 140], [129, 70], 0, 256, "half"),
    (256, "bf16", 128, 128, [150, 3], [140, 3], 70, 32, "adjacent"),
    (256, "bf16", 128, 128, [150], [150], 0, 0, "half"),
    (128, "f32", 256, 32, [90, 64, 5], [64, 64, 5], 0, 128, "half"),
]


@pytest.mark.parametrize("D,dtype,Hq,H,lens,news,window,rot,pairs", ATTEND)
def test_attend(q, D, dtype, Hq, H, lens, news, window, rot, pairs):
    g, raw, table, cu = attend_case(D, H, lens, news, sum(lens) + D)
    Tq = int(cu[-1])
    qx = round_to(g.standard_normal((Tq, Hq, D)) * 1.5, dtype)
    rt = sh.rope_table(g, max(lens) + 8, rot) if rot else None
    pos = g.integers(0, max(lens) + 8, Tq).astype(np.int32) if rot else None
    want, lse, bo, bl = sh.attend(qx, cu, raw, table, lens, D ** -0.5, window, rt, pos, pairs, D, dtype)
    got, gl = run_attend(q, raw, table, cu, lens, qx, D, dtype, window, rt, pos, pairs)
    assert_within(got, want, bo, "out")
    assert_within(gl, lse, bl, "lse")


@pytest.mark.parametrize("D,dtype,rot", [(64, "f32", 64), (64, "bf16", 16), (64, "bf16", 0), (128, "f16", 128),
                                         (128, "bf16", 128), (128, "bf16", 0), (256, "f32", 0)])
@pytest.mark.parametrize("most", [13 * 64, 1025, 32 * 64, 32 * 64 + 1])
def test_attend_middle_lengths(q, D, dtype, rot, most):
    """Sequences of one workgroup a key head, of four waves or eight, and the
    first length that is cut, among shorter ones."""
    H, Hq = 2, 10
    lens, news = [most, 0, 70, most - 300], [1, 0, 3, 2]
    g, raw, table, cu = attend_case(D, H, lens, news, most + D)
    qx = round_to(g.standard_normal((6, Hq, D)), dtype)
    rt = sh.rope_table(g, 100, rot) if rot else None
    pos = g.integers(0, 100, 6).astype(np.int32) if rot else None
    for window in (0, 64 * 14):
        want, lse, bo, bl = sh.attend(qx, cu, raw, table, lens, D ** -0.5, window, rt, pos, "half", D, dtype)
        got, gl = run_attend(q, raw, table, cu, lens, qx, D, dtype, window, rt, pos, "half")
        assert_within(got, want, bo, f"out {window}")
        assert_within(gl, lse, bl, f"lse {window}")


@pytest.mark.parametrize("D,dtype,rot", [(64, "f32", 64), (64, "bf16", 16), (64, "bf16", 0), (128, "f16", 128),
                                         (128, "bf16", 128), (128, "bf16", 0), (256, "f32", 64), (256, "bf16", 256),
                                         (256, "bf16", 0)])
@pytest.mark.parametrize("lens,H,max_len", [([70, 200], 2, 200), ([70, 200], 40, 200), ([70, 200], 66, 900),
                                            ([70, 200], 150, 200), ([1200, 700], 2, 2200), ([1200, 700], 8, 2200),
                                            ([1200, 700, 90, 1], 8, 2200)])
def test_attend_more_and_fewer_heads(q, D, dtype, rot, lens, H, max_len):
    """From a few workgroups, which share a tile's values, to several a compute
    unit; whole and in chunks."""
    news = ([1, 2] + [1] * len(lens))[: len(lens)]
    g, raw, table, cu = attend_case(D, H, lens, news, H + D)
    table = np.concatenate([table, np.full((len(lens), 35), -1, np.int32)], 1)
    Tq = int(cu[-1])
    qx = round_to(g.standard_normal((Tq, 3 * H, D)), dtype)
    rt = sh.rope_table(g, 100, rot) if rot else None
    pos = g.integers(0, 100, Tq).astype(np.int32) if rot else None
    want, lse, bo, bl = sh.attend(qx, cu, raw, table, lens, D ** -0.5, 0, rt, pos, "half", D, dtype)
    got, gl = run_attend(q, raw, table, cu, lens, qx, D, dtype, 0, rt, pos, "half", max_len=max_len)
    assert_within(got, want, bo, "out")
    assert_within(gl, lse, bl, "lse")


@pytest.mark.parametrize("D,dtype,rot", [(64, "f32", 64), (64, "bf16", 16), (64, "bf16", 0), (128, "f16", 128),
                                         (128, "bf16", 128), (128, "bf16", 0), (256, "f32", 64), (256, "bf16", 256),
                                         (256, "bf16", 0)])
@pytest.mark.parametrize("lens,news,H,max_len", [
    ([200, 140], [150, 70], 32, 200),  # tiles of 64 rows, whole
    ([65, 450, 1], [65, 135, 1], 32, 700),
    ([900, 300], [65, 33], 16, 2200),  # in chunks
    ([129, 140], [129, 70], 64, 140),  # of 128 rows
    ([900, 300], [128, 100], 32, 2200),
    ([900, 300], [128, 100], 32, 3200),
])
@pytest.mark.parametrize("window", [0, 100])
def test_attend_prompt_tiles(q, D, dtype, rot, lens, news, H, max_len, window):
    g, raw, table, cu = attend_case(D, H, lens, news, H + D)
    table = np.concatenate([table, np.full((len(lens), 35), -1, np.int32)], 1)
    Tq = int(cu[-1])
    qx = round_to(g.standard_normal((Tq, H, D)), dtype)
    rt = sh.rope_table(g, 100, rot) if rot else None
    pos = g.integers(0, 100, Tq).astype(np.int32) if rot else None
    want, lse, bo, bl = sh.attend(qx, cu, raw, table, lens, D ** -0.5, window, rt, pos, "half", D, dtype)
    got, gl = run_attend(q, raw, table, cu, lens, qx, D, dtype, window, rt, pos, "half", max_len=max_len)
    assert_within(got, want, bo, "out")
    assert_within(gl, lse, bl, "lse")


@pytest.mark.parametrize("D,H,G,n,L,window", [(256, 8, 2, 590, 1994, 1514), (256, 4, 8, 77, 1975, 1523), (128, 2, 4, 100, 9000, 700),
                                              (64, 8, 8, 40, 5000, 2000)])
def test_attend_window_and_the_workspace_without(q, D, H, G, n, L, window):
    """A window that would have another kernel take the call, in chunks, does not
    where the workspace, sized without it, has no room for them."""
    lens, news = [L, 40], [n, 3]
    g, raw, table, cu = attend_case(D, H, lens, news, L)
    qx = round_to(g.standard_normal((n + 3, H * G, D)), "f32")
    want, lse, bo, bl = sh.attend(qx, cu, raw, table, lens, D ** -0.5, window, None, None, "half", D, "f32")
    got, gl = run_attend(q, raw, table, cu, lens, qx, D, "f32", window, None, None, "half")
    assert_within(got, want, bo, "out")
    assert_within(gl, lse, bl, "lse")


def test_attend_large_tiles_in_chunks(q):
    D, H = 64, 128
    lens, news = [800, 100], [100, 70]
    g, raw, table, cu = attend_case(D, H, lens, news, 1)
    table = np.concatenate([table, np.full((2, 35), -1, np.int32)], 1)
    qx = round_to(g.standard_normal((170, H, D)), "f32")
    want, lse, bo, bl = sh.attend(qx, cu, raw, table, lens, D ** -0.5, 0, None, None, "half", D, "f32")
    got, gl = run_attend(q, raw, table, cu, lens, qx, D, "f32", 0, None, None, "half", max_len=2200)
    assert_within(got, want, bo, "out")
    assert_within(gl, lse, bl, "lse")


def test_attend_large_scores(q):
    """Scores in the hundreds, falling and rising along the sequence: the running
    maximum is what keeps the exponentials finite."""
    D, H, Hq = 128, 1, 4
    for sign in (1, -1):
        lens, news = [400], [3]
        g, raw, table, cu = attend_case(D, H, lens, news, 3)
        sc = raw[..., 128 * D:].view(np.float32)
        for i in range(400):
            sc[table[0, i // 64], :, i % 64] = (1 + (i if sign > 0 else 400 - i)) / 2000
        qx = round_to(g.standard_normal((3, Hq, D)) * 4, "f32")
        want, lse, bo, bl = sh.attend(qx, cu, raw, table, lens, D ** -0.5, 0, None, None, "half", D, "f32")
        assert np.abs(lse).max() > 100
        got, gl = run_attend(q, raw, table, cu, lens, qx, D, "f32", 0, None, None, "half")
        assert_within(got, want, bo, "out")
        assert_within(gl, lse, bl, "lse")


def test_attend_values_of_many_sizes(q):
    """Value scales over forty orders of magnitude, the large ones last: what
    the accumulators are counted in has to follow."""
    D, H, Hq = 64, 1, 2
    lens, news = [500], [1]
    g, raw, table, cu = attend_case(D, H, lens, news, 4)
    sc = raw[..., 128 * D:].view(np.float32)
    for i in range(500):
        sc[table[0, i // 64], :, 64 + i % 64] = 10.0 ** (-20 + 40 * i / 500)
    sc[table[0, 0], :, 64: 80] = 0.0
    qx = round_to(g.standard_normal((1, Hq, D)), "f32")
    want, lse, bo, bl = sh.attend(qx, cu, raw, table, lens, D ** -0.5, 0, None, None, "half", D, "f32")
    got, gl = run_attend(q, raw, table, cu, lens, qx, D, "f32", 0, None, None, "half")
    assert_within(got, want, bo, "out")
    assert_within(gl, lse, bl, "lse")


def test_attend_unseen_pages_and_positions(q):
    """A page outside the cache in the middle of a sequence counts as unseen; a
    position outside the table makes its row NaN and no other."""
    D, H, Hq = 128, 2, 4
    lens, news = [300, 70], [4, 2]
    g, raw, table, cu = attend_case(D, H, lens, news, 9)
    table[0, 1], table[0, 3], table[1, 0] = -1, raw.shape[0], 2 ** 31 - 1
    table[1, 1] = -(2 ** 31)  # sequence 1 sees nothing at all
    qx = round_to(g.standard_normal((6, Hq, D)), "f32")
    rt = sh.rope_table(g, 50, D)
    pos = np.array([0, 49, 50, 3, 1, 1], np.int32)
    want, lse, bo, bl = sh.attend(qx, cu, raw, table, lens, D ** -0.5, 0, rt, np.clip(pos, 0, 49), "half", D, "f32")
    assert np.isneginf(lse[4:]).all()
    want[2], lse[2] = np.nan, np.nan
    got, gl = run_attend(q, raw, table, cu, lens, qx, D, "f32", 0, rt, pos, "half")
    assert_within(got, want, np.nan_to_num(bo), "out")
    assert_within(gl, lse, np.nan_to_num(bl), "lse")


def test_attend_looser_maxima(q):
    """max_q and max_len are limits: larger ones change nothing but the split;
    lengths beyond max_len are cut to it, tokens beyond max_q left out."""
    D, H, Hq = 128, 2, 8
    lens, news = [500, 90], [3, 1]
    g, raw, table, cu = attend_case(D, H, lens, news, 21)
    table = np.concatenate([table, np.full((2, 100), -1, np.int32)], 1)
    qx = round_to(g.standard_normal((4, Hq, D)), "f32")
    want, lse, bo, bl = sh.attend(qx, cu, raw, table, lens, D ** -0.5, 0, None, None, "half", D, "f32")
    for max_len, max_q in ((500, 3), (6000, 3), (108 * 64, 6)):
        got, gl = run_attend(q, raw, table, cu, lens, qx, D, "f32", 0, None, None, "half", max_len=max_len, max_q=max_q,
                             extra_rows=2)
        assert_within(got, want, bo, f"out {max_len} {max_q}")
        assert_within(gl, lse, bl, "lse")
    cut = [300, 90]
    want, lse, bo, bl = sh.attend(qx, cu, raw, table, cut, D ** -0.5, 0, None, None, "half", D, "f32")
    got, gl = run_attend(q, raw, table, cu, lens, qx, D, "f32", 0, None, None, "half", max_len=300)
    assert_within(got, want, bo, "out, cut")
    got, gl = run_attend(q, raw, table, cu, lens, qx, D, "f32", 0, None, None, "half", max_len=300, max_q=2)
    assert (got[2] == 7.0).all() and (gl[2] == 7.0).all()
    assert_within(got[[0, 1, 3]], want[[0, 1, 3]], bo[[0, 1, 3]], "out, two tokens")


@pytest.mark.parametrize("D,Hq,n,max_len", [(64, 2, 2, 300), (128, 64, 70, 300), (64, 2, 2, 9000), (128, 64, 70, 2500)])
def test_attend_numbers_out_of_range(q, D, Hq, n, max_len):
    """Bounds and lengths that lie outside what the call's sizes allow are cut to
    it: rows before the first and behind the last, a negative length, one beyond
    the page table."""
    H = Hq // 2
    g, raw, table, cu = attend_case(D, H, [1, 5, 300], [1, 0, n], 17)
    table = np.concatenate([table, np.full((3, 150), -1, np.int32)], 1)
    Tq = int(cu[-1])
    qx = round_to(g.standard_normal((Tq, Hq, D)), "f32")
    cut = [0, 5, max_len]
    want, lse, bo, bl = sh.attend(qx, cu, raw, table, cut, D ** -0.5, 0, None, None, "half", D, "f32")
    odd = np.array([-4, 1, 1, 2 ** 31 - 1], np.int32)
    got, gl = run_attend(q, raw, table, odd, [-(2 ** 31), 5, 2 ** 31 - 1], qx, D, "f32", 0, None, None, "half",
                         max_len=max_len, max_q=n, extra_rows=0)
    assert np.isneginf(gl[0]).all()
    assert_within(got, want, bo, "out")
    assert_within(gl, lse, bl, "lse")


def test_tensors_elsewhere_are_refused(q):
    import torch

    kv = cache_of(q, poisoned_cache(2, 1, 64), 64)
    x = torch.zeros(1, 1, 64, device="cuda")
    with pytest.raises(ValueError):
        q.q8k_kv_read(q.Q8K_F32, kv, torch.zeros(1, dtype=torch.int32), 1, x, x.clone())
    with pytest.raises(ValueError):
        q.q8k_kv_read(q.Q8K_F32, kv, torch.zeros(1, dtype=torch.int32, device="cuda"), 1, x, x.cpu())


@pytest.mark.parametrize("B,D,H,Hq,window", [(70, 64, 1, 2, 0), (130, 128, 2, 2, 0), (257, 64, 1, 1, 0), (90, 64, 1, 4, 150)])
def test_attend_many_sequences(q, B, D, H, Hq, window):
    """Mixed lengths of more sequences than a wave has lanes, few enough and too
    many to be split, with limits far above the lengths."""
    g = np.random.default_rng(B)
    lens = [int(n) for n in g.integers(0, 300, B)]
    lens[B // 2], lens[B - 1], lens[3] = 6000, 3000, 0
    news = [int(n) for n in g.integers(0, 3, B)]
    news[B // 2] = 2
    g, raw, table, cu = attend_case(D, H, lens, news, B + 1)
    table = np.concatenate([table, np.full((B, 400), -1, np.int32)], 1)
    qx = round_to(g.standard_normal((int(cu[-1]), Hq, D)), "f32")
    want, lse, bo, bl = sh.attend(qx, cu, raw, table, lens, D ** -0.5, window, None, None, "half", D, "f32")
    got, gl = run_attend(q, raw, table, cu, lens, qx, D, "f32", window, None, None, "half", max_len=25000, max_q=5)
    assert_within(got, want, bo, "out")
    assert_within(gl, lse, bl, "lse")


@pytest.mark.parametrize("B,D,H,Hq,max_len", [(130, 64, 1, 2, 2600), (256, 128, 2, 2, 2600), (65, 256, 1, 1, 2000),
                                              (64, 64, 32, 32, 2100), (63, 128, 33, 33, 2100)])
def test_attend_many_sequences_of_long_limits(q, B, D, H, Hq, max_len):
    """Chunks found among more than 64 sequences, some of them cut; and whole
    tiles taken by length, equal lengths among them."""
    g = np.random.default_rng(B + D)
    lens = [int(v) for v in g.integers(0, 150, B)]
    news = [min(v, 1 + v % 2) for v in lens]
    lens[1], lens[B // 2], lens[B - 1] = (2500, 1300, 700) if H < 8 and D < 256 else (700, 150, 700) if H < 8 else (140, 300, 140)
    news[1] = news[B // 2] = news[B - 1] = 1
    g, raw, table, cu = attend_case(D, H, lens, news, B)
    table = np.concatenate([table, np.full((B, 41), -1, np.int32)], 1)
    qx = round_to(g.standard_normal((int(cu[-1]), Hq, D)), "f32")
    want, lse, bo, bl = sh.attend(qx, cu, raw, table, lens, D ** -0.5, 0, None, None, "half", D, "f32")
    got, gl = run_attend(q, raw, table, cu, lens, qx, D, "f32", 0, None, None, "half", max_len=max_len, max_q=2)
    assert_within(got, want, bo, "out")
    assert_within(gl, lse, bl, "lse")


def test_attend_far_pages(q):
    """Pages beyond 4 GiB of the cache."""
    import torch

    D, H, Hq = 64, 2, 2
    rec = record(D)
    pages = (5 << 30) // (rec * H)
    lens, news = [100], [1]
    g, raw, table, cu = attend_case(D, H, lens, news, 8)
    big = torch.empty(pages * H * rec, dtype=torch.uint8, device="cuda")
    small = raw.shape[0]
    at = pages - small
    big[at * H * rec:] = to_dev(raw).reshape(-1)
    kv = q.KVCache(big, pages, H, D)
    qx = round_to(g.standard_normal((1, Hq, D)), "f32")
    want, lse, bo, bl = sh.attend(qx, cu, raw, table, lens, D ** -0.5, 0, None, None, "half", D, "f32")
    out, ls = torch.zeros(1, Hq, D, device="cuda"), torch.zeros(1, Hq, device="cuda")
    far = np.where((table >= 0) & (table < small), table + at, table).astype(np.int32)
    q.qattend(q.Q8K_F32, to_dev_as(qx, "f32"), Hq * D, Hq, kv, 1, to_dev(cu), 1, 1, to_dev(far), far.shape[1],
              to_dev(np.array(lens, np.int32)), 100, D ** -0.5, 0, None, None, out, ls)
    assert_within(back(out), want, bo, "out")
    # and an append there
    slot = np.array([pages * 64 - 1], np.int32)
    x = g.standard_normal((1, 2 * H, D)).astype(np.float32)
    xd = to_dev(x)
    q.q8k_kv_append(q.Q8K_F32, xd[:, :H], 2 * H * D, xd[:, H:], 2 * H * D, 1, None, None, to_dev(slot), kv)
    kd, vd = torch.zeros(1, H, D, device="cuda"), torch.zeros(1, H, D, device="cuda")
    q.q8k_kv_read(q.Q8K_F32, kv, to_dev(slot), 1, kd, vd)
    for got, part in ((kd, x[:, :H]), (vd, x[:, H:])):
        c, s = sh.quantise(part)
        assert_exact(back(got), c.astype(np.float32) * s[..., None], "far slot")


# -------------------------------------------------------------------- logprobs
def run_logprobs(q, x, dtype, targets, n, stride=None, offset=0):
    """x fp32 [T][V] of the type's values -> host results, from rows `stride` apart that start `offset` elements in."""
    import torch

    T, V = x.shape
    stride = stride or V
    flat = torch.full((T * stride + offset,), float("inf"), dtype=torch_dtype(dtype), device="cuda")
    view = flat[offset:].as_strided((T, V), (stride, 1), flat.storage_offset() + offset)
    view.copy_(to_dev_as(x, dtype))
    nan = lambda *s: torch.full(s, float("nan"), device="cuda")  # noqa: E731
    r = dict(logprob=nan(T), entropy=nan(T), lse=nan(T), top_logprob=nan(T, n),
             top_ids=torch.full((T, n), -7, dtype=torch.int32, device="cuda"))
    need = q.qlogprobs_workspace_bytes(T, V, n)
    q.qlogprobs(q_dtype(q, dtype), view, stride, T, V, to_dev(targets), r["logprob"], r["entropy"], r["lse"], n,
                r["top_ids"] if n else None, r["top_logprob"] if n else None, poisoned(need) if need else None, need)
    return {k: host(v) for k, v in r.items()}


def check_logprobs(got, want, what=""):
    for k in ("logprob", "lse", "entropy", "top_logprob"):
        assert_within(got[k], want[k][0], want[k][1], f"{what} {k}")
    if want["top_ids"].size:
        assert_exact(got["top_ids"], want["top_ids"], f"{what} top ids")


@pytest.mark.parametrize("V,n", [(1, 1), (2, 2), (5, 0), (31, 31), (33, 32), (255, 3), (256, 20), (1000, 32),
                                 (8191, 5), (8192, 1), (8193, 32), (32000, 8),
                                 (32769, 1), (70001, 20), (131072, 0)])
@pytest.mark.parametrize("dtype", sh.DTYPES)
def test_logprobs(q, V, n, dtype):
    T = 3
    g = np.random.default_rng(V)
    x = g.standard_normal((T, V)) * 3
    x[:, g.integers(0, V, 4)] += 12
    if V > 40:
        x[1, V // 2: V // 2 + V // 4] = -np.inf
    x = round_to(x, dtype)
    targets = np.array([0, V - 1, V // 2], np.int32)
    got = run_logprobs(q, x, dtype, targets, n, stride=V + 3 if V % 2 else None, offset=V % 8)
    check_logprobs(got, sh.logprobs(x, targets, n), f"{V} {dtype}")


def test_logprobs_many_rows(q):
    g = np.random.default_rng(0)
    x = round_to(g.standard_normal((300, 9000)) * 2, "bf16")
    targets = g.integers(-1, 9001, 300).astype(np.int32)  # some outside the vocabulary: NaN
    check_logprobs(run_logprobs(q, x, "bf16", targets, 4), sh.logprobs(x, targets, 4))


def test_logprobs_long_rows_whole(q):
    """More rows than are cut into parts: one workgroup goes through a row in
    several rounds, here with the largest last, first and in the middle."""
    T, V, n = 260, 66000, 20
    g = np.random.default_rng(17)
    x = g.standard_normal((T, V)).astype(np.float32)
    x += np.linspace(-3, 3, V, dtype=np.float32) * g.integers(-1, 2, (T, 1))
    x[5] = -np.inf
    x[5, 40000:40007] = 1.0
    x[6, 33000:] = -np.inf
    x = round_to(x, "f16")
    t = g.integers(0, V, T).astype(np.int32)
    check_logprobs(run_logprobs(q, x, "f16", t, n), sh.logprobs(x, t, n))


@pytest.mark.parametrize("V", [40, 10007, 80000])
def test_logprobs_ties(q, V):
    """Equal logits everywhere, in stretches, and as +0 and -0: the lowest ids."""
    g = np.random.default_rng(1)
    x = np.zeros((5, V), np.float32)
    x[1] = -0.0
    x[1, ::3] = 0.0
    x[2] = g.integers(-2, 3, V)
    x[3, V // 2:] = 1.0
    x[4] = -np.inf
    x[4, [3, V - 1]] = -5.0  # fewer finite logits than alternatives
    t = np.array([1, 2, 3, V - 1, 0], np.int32)
    check_logprobs(run_logprobs(q, x, "f32", t, 32), sh.logprobs(x, t, 32))


def test_logprobs_rows_of_nothing_and_infinities(q):
    V, n = 9001, 3
    g = np.random.default_rng(2)
    x = g.standard_normal((4, V)).astype(np.float32)
    x[0] = -np.inf
    x[1, 77] = np.inf
    x[2, 5] = np.nan
    t = np.array([4, 77, 8, 9], np.int32)
    got = run_logprobs(q, x, "f32", t, n)
    want = sh.logprobs(x[[0, 3]], t[[0, 3]], n)
    assert np.isneginf(want["lse"][0][0]) and want["entropy"][0][0] == 0
    check_logprobs({k: v[[0, 3]] for k, v in got.items()}, want)
    for r in (1, 2):
        for k in ("logprob", "lse", "entropy"):
            assert np.isnan(got[k][r])
        assert np.isnan(got["top_logprob"][r]).all()
    assert got["top_ids"][1][0] == 77
    rest = x[2].copy()
    rest[5] = -np.inf
    assert_exact(got["top_ids"][2], np.argsort(-rest, kind="stable")[:n].astype(np.int32), "ids beside a NaN")


def test_logprobs_sharp_rows(q):
    """One logit far above all others, and very negative ones."""
    V = 20000
    g = np.random.default_rng(3)
    x = (g.standard_normal((3, V)) * 2).astype(np.float32)
    x[0, 123] = 60.0
    x[1] -= 3e4
    x[2, 7], x[2, 8] = 1e30, -1e30
    t = np.array([123, 5, 8], np.int32)
    check_logprobs(run_logprobs(q, x, "f32", t, 2), sh.logprobs(x, t, 2))


# ------------------------------------------------------------- a step together
def _weights(q, g, rows, K):
    import synth

    return to_dev(synth.q4k_weights(g, rows, K, d_range=(1e-5, 1e-4), dmin_range=(0.0, 1e-4)))


def test_model_step(q):
    """A prompt and two decode steps through the projections, the cache, the
    attention and the output head, every stage checked on what the stage before
    left: q|k|v is one fused weight, whose output's slices go into the cache and
    the attention as they lie."""
    import torch

    g = np.random.default_rng(30)
    hidden, Hq, H, D, V = 512, 4, 2, 128, 1003
    qkv_rows = (Hq + 2 * H) * D
    wqkv, wo, wh = _weights(q, g, qkv_rows, hidden), _weights(q, g, hidden, Hq * D), _weights(q, g, V, hidden)
    pages, n0 = 6, 130
    order = g.permutation(pages).astype(np.int32)
    table = order[None, :4].copy()
    rt = sh.rope_table(g, 256, D)
    rope, tabled = rope_of(q, rt, "half"), to_dev(table)
    mirror = poisoned_cache(pages, H, D)
    kv = cache_of(q, mirror, D)
    slot_of = lambda p: (order[p // 64] * 64 + p % 64).astype(np.int32)  # noqa: E731
    f32 = dict(dtype=torch.float32, device="cuda")

    def step(x, first):
        n = x.shape[0]
        xd = to_dev(x)
        qkv = torch.full((n, Hq + 2 * H, D), float("nan"), **f32)
        xq = poisoned(q.q8k_act_bytes(n, hidden))
        if n == 1:
            q.qmatvec_f32(q.Q8K_Q4_K, wqkv, qkv_rows, hidden, xd, 1, qkv)
        else:
            q.q8k_pack(xd, n, hidden, xq)
            wsb = q.qmatmul_prefill_workspace_bytes(q.Q8K_Q4_K, qkv_rows, hidden, n)
            q.qmatmul_prefill(q.Q8K_Q4_K, wqkv, qkv_rows, hidden, xq, n, qkv, poisoned(wsb), wsb)
        p = first + np.arange(n)
        pos, slots = to_dev(p.astype(np.int32)), to_dev(slot_of(p))
        q.q8k_kv_append(q.Q8K_F32, qkv[:, Hq: Hq + H], qkv_rows, qkv[:, Hq + H:], qkv_rows, n, pos, rope, slots, kv)
        rows = host(qkv)
        sh.append(mirror, rows[:, Hq: Hq + H], rows[:, Hq + H:], rt, p, "half", slot_of(p), D)
        assert_exact(cache_bytes(kv, pages, H, D), mirror, "cache")
        out, lse = torch.full((n, Hq, D), float("nan"), **f32), torch.full((n, Hq), float("nan"), **f32)
        cu, lens = np.array([0, n], np.int32), np.array([first + n], np.int32)
        need = q.qattend_workspace_bytes(kv, Hq, 1, n, n, 256)
        ws = poisoned(need)
        q.qattend(q.Q8K_F32, qkv, qkv_rows, Hq, kv, 1, to_dev(cu), n, n, tabled, 4, to_dev(lens), 256, D ** -0.5, 0, pos,
                  rope, out, lse, ws, need)
        want, wl, bo, bl = sh.attend(rows[:, :Hq], cu, mirror, table, lens, D ** -0.5, 0, rt, p, "half", D, "f32")
        assert_within(host(out), want, bo, "attention")
        assert_within(host(lse), wl, bl, "lse")
        last = out[-1:].reshape(1, Hq * D).contiguous()
        h = torch.full((1, hidden), float("nan"), **f32)
        q.qmatvec_f32(q.Q8K_Q4_K, wo, hidden, Hq * D, last, 1, h)
        logits = torch.full((1, V), float("nan"), **f32)
        q.qmatvec_f32(q.Q8K_Q4_K, wh, V, hidden, h, 1, logits)
        x = host(logits)
        t = np.array([5], np.int32)
        r = dict(logprob=torch.zeros(1, **f32), entropy=torch.zeros(1, **f32), lse=torch.zeros(1, **f32),
                 top_logprob=torch.zeros(1, 5, **f32), top_ids=torch.zeros(1, 5, dtype=torch.int32, device="cuda"))
        need = q.qlogprobs_workspace_bytes(1, V, 5)
        q.qlogprobs(q.Q8K_F32, logits, V, 1, V, to_dev(t), r["logprob"], r["entropy"], r["lse"], 5, r["top_ids"],
                    r["top_logprob"], poisoned(need), need)
        check_logprobs({k: host(v) for k, v in r.items()}, sh.logprobs(x, t, 5), "step")

    step(g.standard_normal((n0, hidden)).astype(np.float32), 0)
    step(g.standard_normal((1, hidden)).astype(np.float32), n0)
    step(g.standard_normal((1, hidden)).astype(np.float32), n0 + 1)


def test_graphs_share_a_workspace(q):
    """Two captured decode steps on one workspace, replayed in turn with eager
    calls between them: every replay gives the eager results, bit for bit, on
    inputs that change from replay to replay."""
    import torch

    D, H, Hq, V, n = 128, 2, 8, 9100, 4
    g = np.random.default_rng(12)
    cases = []
    for lens in ([900, 64], [2000, 1]):
        _, raw, table, cu = attend_case(D, H, lens, [1, 1], sum(lens))
        c = dict(kv=cache_of(q, raw, D), table=to_dev(table), cu=to_dev(cu), lens=to_dev(np.array(lens, np.int32)),
                 most=table.shape[1], len=max(lens), slots=to_dev((table[[0, 1], [(l - 1) // 64 for l in lens]] * 64
                                                                   + [(l - 1) % 64 for l in lens]).astype(np.int32)),
                 row=torch.zeros(2, Hq + 2 * H, D, device="cuda"), logits=torch.zeros(2, V, device="cuda"),
                 pos=to_dev(np.array(lens, np.int32) - 1))
        f32 = dict(dtype=torch.float32, device="cuda")
        c["res"] = [torch.zeros(2, Hq, D, **f32), torch.zeros(2, Hq, **f32), torch.zeros(2, **f32),
                    torch.zeros(2, **f32), torch.zeros(2, **f32), torch.zeros(2, n, dtype=torch.int32, device="cuda"),
                    torch.zeros(2, n, **f32)]
        cases.append(c)
    rope = rope_of(q, sh.rope_table(g, 2000, D), "adjacent")
    targets = to_dev(np.array([3, 9099], np.int32))
    need = max([q.qattend_workspace_bytes(c["kv"], Hq, 2, 2, 1, c["len"]) for c in cases]
               + [q.qlogprobs_workspace_bytes(2, V, n)])
    ws = poisoned(need)

    def step(c, res):
        st = (Hq + 2 * H) * D
        q.q8k_kv_append(q.Q8K_F32, c["row"][:, Hq: Hq + H], st, c["row"][:, Hq + H:], st, 2, c["pos"], rope, c["slots"],
                        c["kv"])
        q.qattend(q.Q8K_F32, c["row"], st, Hq, c["kv"], 2, c["cu"], 2, 1, c["table"], c["most"], c["lens"], c["len"],
                  D ** -0.5, 0, c["pos"], rope, res[0], res[1], ws, need)
        q.qlogprobs(q.Q8K_F32, c["logits"], V, 2, V, targets, res[2], res[3], res[4], n, res[5], res[6], ws, need)

    graphs = []
    for c in cases:
        step(c, c["res"])
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=s):
            step(c, c["res"])
        graphs.append(gr)
    for rep in range(4):
        for c, gr in zip(cases, graphs):
            c["row"].copy_(to_dev(g.standard_normal((2, Hq + 2 * H, D)).astype(np.float32)))
            c["logits"].copy_(to_dev(g.standard_normal((2, V)).astype(np.float32) * 3))
            for r in c["res"]:
                r.fill_(-1)
            gr.replay()
            torch.cuda.synchronize()
            got = [host(r) for r in c["res"]]
            eager = [torch.zeros_like(r) for r in c["res"]]
            step(c, eager)
            for a, b in zip(got, eager):
                assert np.array_equal(a.view(np.uint32), host(b).view(np.uint32)), rep


def test_other_streams(q):
    """Calls on a side stream, given by argument or as torch's current one."""
    import torch

    D, H, Hq = 64, 1, 4
    lens, news = [1500], [1]
    g, raw, table, cu = attend_case(D, H, lens, news, 2)
    qx = round_to(g.standard_normal((1, Hq, D)), "f32")
    want, lse, bo, bl = sh.attend(qx, cu, raw, table, lens, D ** -0.5, 0, None, None, "half", D, "f32")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got, gl = run_attend(q, raw, table, cu, lens, qx, D, "f32", 0, None, None, "half")
    assert_within(got, want, bo, "out")
    kv = cache_of(q, raw, D)
    slots = to_dev(table[0, :1] * 64)
    kd, vd = torch.zeros(1, H, D, device="cuda"), torch.zeros(1, H, D, device="cuda")
    torch.cuda.synchronize()
    q.q8k_kv_read(q.Q8K_F32, kv, slots, 1, kd, vd, s)
    s.synchronize()
    k, ks, _, _ = sh.held(raw, host(slots), D)
    assert_exact(host(kd), k.astype(np.float32) * ks[..., None], "keys")


def test_results_repeat(q):
    """The same call twice gives the same bits (no order of arrival decides a sum)."""
    D, H, Hq = 128, 2, 8
    lens, news = [6000, 300], [1, 1]
    g, raw, table, cu = attend_case(D, H, lens, news, 6)
    qx = round_to(g.standard_normal((2, Hq, D)), "f32")
    a = run_attend(q, raw, table, cu, lens, qx, D, "f32", 0, None, None, "half")
    b = run_attend(q, raw, table, cu, lens, qx, D, "f32", 0, None, None, "half")
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])
    x = round_to(g.standard_normal((9, 30000)), "f32")
    t = np.zeros(9, np.int32)
    a, b = run_logprobs(q, x, "f32", t, 7), run_logprobs(q, x, "f32", t, 7)
    assert all(np.array_equal(a[k], b[k]) for k in a)


@pytest.mark.parametrize("D,dtype,H,Hq,n", [(128, "f32", 2, 8, 1), (64, "bf16", 1, 16, 2), (128, "bf16", 16, 32, 60)])
def test_captured_step_as_sequences_grow(q, D, dtype, H, Hq, n):
    """One captured call serves whatever lengths lie on the device when it is
    replayed, up to the limit that it was captured for."""
    import torch

    B, most = 2, 4480
    g, raw, table, cu = attend_case(D, H, [most, most], [n, n], D + n)
    kv, tabled, cud = cache_of(q, raw, D), to_dev(table), to_dev(cu)
    lens = to_dev(np.array([n, n], np.int32))
    qx = round_to(g.standard_normal((B * n, Hq, D)), dtype)
    qd = to_dev_as(qx, dtype)
    out = torch.zeros(B * n, Hq, D, dtype=torch_dtype(dtype), device="cuda")
    lse = torch.zeros(B * n, Hq, device="cuda")
    need = q.qattend_workspace_bytes(kv, Hq, B, B * n, n, most)
    ws = poisoned(need)

    def call(o, l):
        q.qattend(q_dtype(q, dtype), qd, Hq * D, Hq, kv, B, cud, B * n, n, tabled, table.shape[1], lens, most, D ** -0.5,
                  0, None, None, o, l, ws, need)

    call(out, lse)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        call(out, lse)
    for now in ([n, n + 3], [2100, 64 + n], [most, 700], [most, most]):
        lens.copy_(to_dev(np.array(now, np.int32)))
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        got, gl = back(out), back(lse)
        want, wl, bo, bl = sh.attend(qx, cu, raw, table, now, D ** -0.5, 0, None, None, "half", D, dtype)
        assert_within(got, want, bo, f"out {now}")
        assert_within(gl, wl, bl, f"lse {now}")
        o, l = torch.zeros_like(out), torch.zeros_like(lse)
        call(o, l)
        assert np.array_equal(back(o), got) and np.array_equal(back(l), gl)


def test_two_calls_at_once(q):
    """Calls on two streams, each with its own workspace."""
    import torch

    D, H, Hq = 128, 4, 8
    cases = []
    for seed, lens in ((1, [5000, 900]), (2, [300, 4000])):
        g, raw, table, cu = attend_case(D, H, lens, [1, 1], seed)
        qx = round_to(g.standard_normal((2, Hq, D)), "f32")
        kv = cache_of(q, raw, D)
        need = q.qattend_workspace_bytes(kv, Hq, 2, 2, 1, max(lens))
        cases.append(dict(kv=kv, table=to_dev(table), most=table.shape[1], cu=to_dev(cu), lens=to_dev(np.array(lens, np.int32)),
                          n=max(lens), q=to_dev(qx), out=torch.zeros(2, Hq, D, device="cuda"), need=need, ws=poisoned(need),
                          lse=torch.zeros(2, Hq, device="cuda"), s=torch.cuda.Stream(),
                          want=sh.attend(qx, cu, raw, table, lens, D ** -0.5, 0, None, None, "half", D, "f32")))
    torch.cuda.synchronize()
    for _ in range(20):
        for c in cases:
            q.qattend(q.Q8K_F32, c["q"], Hq * D, Hq, c["kv"], 2, c["cu"], 2, 1, c["table"], c["most"], c["lens"], c["n"],
                      D ** -0.5, 0, None, None, c["out"], c["lse"], c["ws"], c["need"], c["s"])
    for c in cases:
        c["s"].synchronize()
        want, wl, bo, bl = c["want"]
        assert_within(host(c["out"]), want, bo, "out")
        assert_within(host(c["lse"]), wl, bl, "lse")


@pytest.mark.parametrize("n", [2, 200])
def test_attend_nothing_cached(q, n):
    """A limit of no tokens at all: every row is one that sees nothing."""
    for D, H, Hq in ((64, 1, 3), (128, 64, 64), (256, 2, 2)):
        g, raw, table, cu = attend_case(D, H, [0, 0], [n, 1], 1)
        qx = round_to(g.standard_normal((n + 1, Hq, D)), "f32")
        got, gl = run_attend(q, raw, table, cu, [0, 0], qx, D, "f32", 0, None, None, "half")
        assert_exact(got, np.zeros_like(got), "out")
        assert np.isneginf(gl).all()
