"""What the binding sees of the tensors that it is given and the C side cannot:
where their rows lie.  On the CPU: calls that have nothing to do (a cache without
pages, no sequence) go through all checks and enqueue nothing."""
import pytest
import torch

from test_serving_abi import A16, app, att, kv, lps, q  # noqa: F401  (q is the fixture)

H, D = 2, 64  # of the cache that app() and att() use


def append(q, k, stride, T, what="k"):
    args = dict(k=k, ks=stride) if what == "k" else dict(v=k, vs=stride)
    app(q, T=T, cache=kv(q, pages=0), **args)


def attend(q, x, stride, T, heads=4):
    att(q, qp=x, qs=stride, heads=heads, B=0, Tq=T)


def logprobs(q, x, stride, T, V):
    with pytest.raises(q.Q8KError, match="logprob"):  # behind the binding's checks
        lps(q, x=x, stride=stride, T=T, V=V, lp=None)


def views():
    """(tensor, stride, rows) that hold rows of 2 heads of 64 values."""
    row = torch.zeros(9, 6, D)
    return [
        (row[:, 2:4], 6 * D, 9), (row[:, 4:], 6 * D, 9), (row, 6 * D, 9), (row[:1, 2:4], 6 * D, 1), (row[2:3, 2:4], 136, 1),
        (row[3:, 2:4], 6 * D, 6), (row[::2, 2:4], 12 * D, 5), (row[:, 2:4], 12 * D, 5),
        (torch.zeros(9, H, D), H * D, 9), (torch.zeros(9, H * D), H * D, 9), (torch.zeros(9 * H * D), H * D, 9),
        (torch.zeros(9 * H * D), 3 * H * D, 3), (torch.zeros(3, 3, H, D), H * D, 9), (torch.zeros(3, 3, H, D), 3 * H * D, 3),
        (torch.zeros(3, 3, 6, D)[:, :, 2:4], 6 * D, 9), (torch.zeros(1, 9, H, D), H * D, 9),
        (torch.zeros(9, 1, H, D), H * D, 9), (torch.zeros(27, H * D), 3 * H * D, 9), (torch.zeros(9, 6, D)[:, 2:4].unsqueeze(1), 6 * D, 9),
        (torch.zeros(9, 6 * D)[:, 2 * D: 4 * D], 6 * D, 9), (torch.zeros(9, 6 * D)[:, 8: 8 + 2 * D], 6 * D, 9),
    ]


@pytest.mark.parametrize("i", range(len(views())))
def test_rows_are_taken(q, i):
    t, stride, T = views()[i]
    append(q, t, stride, T)
    append(q, t, stride, T, "v")
    attend(q, t, stride, T, heads=2)
    logprobs(q, t, stride, T, H * D)


def odd_views():
    row = torch.zeros(9, 6, D)
    return [
        (torch.zeros(9, D, H).transpose(1, 2), H * D, 9),  # a head's values apart
        (torch.zeros(9, H, 2 * D)[..., ::2], 2 * H * D, 9),
        (torch.zeros(9, H, 2 * D)[..., :D], 2 * H * D, 9),  # heads apart
        (torch.zeros(H, 9, D).transpose(0, 1), H * D, 9),  # tokens inside heads
        (torch.zeros(H, 9, D).transpose(0, 1), D, 9),
        (row[:, 2:4], 2 * D, 9), (row[:, 2:4], 5 * D, 9), (row[:, 2:4], 7 * D, 9),  # another stride than the tensor's
        (row, 2 * D, 9), (row, 4 * D, 9), (torch.zeros(9, H * D), H * D + 8, 9),
        (row[::2, 2:4], 6 * D, 5),
        (torch.zeros(1, H, D).expand(9, H, D), H * D, 9),
        (torch.zeros(4, 3, 6, D)[:, :2, 2:4], 6 * D, 8),  # two of three tokens, again and again
        (row[:1, 1:2].expand(1, 2, D), 6 * D, 1),
    ]


@pytest.mark.parametrize("i", range(len(odd_views())))
def test_rows_elsewhere_are_refused(q, i):
    t, stride, T = odd_views()[i]
    for call in (lambda: append(q, t, stride, T), lambda: append(q, t, stride, T, "v"), lambda: attend(q, t, stride, T, 2),
                 lambda: logprobs(q, t, stride, T, H * D)):
        with pytest.raises(ValueError, match="does not hold .* rows of 128 values"):
            call()


def i32(*n):
    return torch.zeros(*n, dtype=torch.int32)


def short(name, need, call):
    with pytest.raises(ValueError, match=f"{name} has {need - 1} elements, {need} are needed"):
        call(need - 1)
    call(need)
    call(need + 3)


def test_short_tensors_are_refused(q):
    """One element less than the call reads or writes, and the same call with all of them."""
    none = kv(q, pages=0)  # appends nothing
    short("slots", 5, lambda n: app(q, T=5, slots=i32(n), cache=none))
    rope = q.Rope(torch.zeros(8, 64), 8, 64)
    short("pos", 5, lambda n: app(q, T=5, pos=i32(n), rope=rope, cache=none))
    app(q, T=5, pos=i32(2), cache=none)  # no rotation: not read

    def read_one(name, n):
        a = dict(slots=A16, k=A16, v=A16)
        a[name] = i32(n) if name == "slots" else torch.zeros(n)
        try:
            q.q8k_kv_read(q.Q8K_F32, kv(q, dim=32), a["slots"], 5, a["k"], a["v"], 0)
        except q.Q8KError as e:  # behind the binding's checks
            assert "head_dim" in str(e)

    short("slots", 5, lambda n: read_one("slots", n))
    for name in ("k", "v"):
        short(name, 5 * 2 * 32, lambda n: read_one(name, n))

    def attend_one(**a):
        try:
            att(q, **{**dict(B=3, Tq=7, max_q=1, max_pages=4, max_len=300), **a})
        except q.Q8KError as e:  # behind the binding's checks
            assert "max_len=300" in str(e)

    short("cu_q", 4, lambda n: attend_one(cu=i32(n)))
    short("kv_len", 3, lambda n: attend_one(lens=i32(n)))
    short("page_table", 12, lambda n: attend_one(table=i32(n)))
    short("pos", 7, lambda n: attend_one(pos=i32(n), rope=rope))
    attend_one(pos=i32(1))
    short("out", 7 * 4 * 64, lambda n: attend_one(out=torch.zeros(n)))
    short("lse", 7 * 4, lambda n: attend_one(lse=torch.zeros(n)))
    short("ws", 1000, lambda n: attend_one(ws=torch.zeros(n, dtype=torch.uint8), wsb=1000))
    short("ws", 250, lambda n: attend_one(ws=torch.zeros(n), wsb=1000))
    short("ws", 251, lambda n: attend_one(ws=torch.zeros(n), wsb=1001))

    def logprobs_one(**a):
        try:
            lps(q, **{**dict(T=5, V=100, stride=99, n=3, ids=A16, tl=A16), **a})
        except q.Q8KError as e:
            assert "stride=99" in str(e)

    for name, arg in (("targets", "targets"), ("logprob", "lp"), ("entropy", "ent"), ("lse", "lse")):
        short(name, 5, lambda n: logprobs_one(**{arg: i32(n) if name == "targets" else torch.zeros(n)}))
    short("top_ids", 15, lambda n: logprobs_one(ids=i32(n)))
    short("top_logprob", 15, lambda n: logprobs_one(tl=torch.zeros(n)))
    short("ws", 64, lambda n: logprobs_one(ws=torch.zeros(n, dtype=torch.uint8), wsb=64))


@pytest.mark.parametrize("i", range(len(views())))
def test_too_few_rows_are_refused(q, i):
    t, stride, T = views()[i]
    more = T + 1
    for call in (lambda: append(q, t, stride, more), lambda: append(q, t, stride, more, "v"),
                 lambda: attend(q, t, stride, more, 2), lambda: logprobs(q, t, stride, more, H * D)):
        with pytest.raises(ValueError, match=f"does not hold {more} rows of 128 values"):
            call()


def test_a_last_row_cut_off(q):
    buf = torch.zeros(3 * 384 + 127)
    with pytest.raises(ValueError, match="does not hold 4 rows"):
        append(q, buf, 384, 4)
    append(q, torch.zeros(3 * 384 + 128), 384, 4)
    with pytest.raises(ValueError, match="does not hold 1 rows"):
        append(q, torch.zeros(127), 384, 1)
    append(q, torch.zeros(1, 2, 64), 384, 0)
    with pytest.raises(q.Q8KError, match="T=-1"):
        append(q, torch.zeros(1, 2, 64), 384, -1)
