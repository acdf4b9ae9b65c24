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
        with pytest.raises(ValueError, match="does not hold rows of 128 values"):
            call()
