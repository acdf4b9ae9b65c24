"""Calls of more threads than a launch can count (2^32) are refused by name."""
from test_serving_abi import A16, app, att, kv, lps, q, refused  # noqa: F401  (q is the fixture)

M = 1 << 24  # the most tokens, or rows, of a call


def test_append_and_read(q):
    c = kv(q, heads=32)
    assert "2^32" in refused(q, "Q8K_ERR_SHAPE", lambda: app(q, T=M, ks=2048, vs=2048, cache=c))
    assert "2^32" in refused(q, "Q8K_ERR_SHAPE", lambda: q.q8k_kv_read(0, c, A16, M, A16, A16, 0))
    app(q, T=M, ks=2048, vs=2048, cache=kv(q, heads=16, pages=0))  # half as many: nothing else to refuse
    app(q, T=M - 32, ks=2048, vs=2048, cache=kv(q, heads=31, pages=0))


def test_attend(q):
    c = kv(q, heads=16)
    big = dict(cache=c, heads=16, qs=1024)
    assert "2^32" in refused(q, "Q8K_ERR_SHAPE", lambda: att(q, B=1 << 20, Tq=1 << 20, max_q=1, **big))
    # 128-row tiles: 64 of them a head and sequence
    assert "2^32" in refused(q, "Q8K_ERR_SHAPE", lambda: att(q, B=1 << 14, Tq=1 << 14, max_q=8192, **big))


def test_logprobs(q):
    assert "2^32" in refused(q, "Q8K_ERR_SHAPE", lambda: lps(q, T=M, V=1, stride=1))
    assert "2^32" in refused(q, "Q8K_ERR_SHAPE", lambda: lps(q, T=M, V=8192, stride=8192))
    assert "2^32" in refused(q, "Q8K_ERR_SHAPE", lambda: lps(q, T=M // 4, V=8193, stride=8193))
