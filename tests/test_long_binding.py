"""The binding's calls of the caches of 8 and of 4 bits on the CPU: each is one Python
frame that calls its checks itself, has its own name, and takes its own cache alone."""
import inspect
import sys

import pytest

from test_serving_abi import A16, q  # noqa: F401  (q is the fixture)


def args_of(q, name):  # noqa: F811
    """Arguments of a call that has nothing to do."""
    kv = q.KVCache(A16, 4, 2, 64, bits=4 if "kv4" in name else 8)
    if "append" in name:
        return 0, A16, 128, A16, 128, 0, None, None, A16, kv, 0
    if "read" in name:
        return 0, kv, A16, 0, A16, A16, 0
    return 0, A16, 256, 4, kv, 0, A16, 0, 0, A16, 4, A16, 200, 0.1, 0, None, None, A16, None, A16, 1 << 30, 0


NAMES = ["q8k_kv_append", "q8k_kv4_append", "q8k_kv_read", "q8k_kv4_read", "qattend", "qattend_kv4"]


@pytest.mark.parametrize("name", NAMES)
def test_a_call_is_one_frame(q, name):  # noqa: F811
    call, args, depths = getattr(q, name), args_of(q, name), []

    def note(frame, event, arg):
        if event == "call" and frame.f_code.co_name == "_check":
            depth = 0
            while frame.f_back is not here:
                frame, depth = frame.f_back, depth + 1
            depths.append(depth)

    here = sys._getframe()
    sys.setprofile(note)
    try:
        call(*args)
    finally:
        sys.setprofile(None)
    assert depths == [1]


@pytest.mark.parametrize("a,b", [NAMES[:2], NAMES[2:4], NAMES[4:]])
def test_names_and_arguments(q, a, b):  # noqa: F811
    f, g = getattr(q, a), getattr(q, b)
    assert f.__name__ == a and g.__name__ == b and f is not g
    assert inspect.signature(f) == inspect.signature(g)
    assert a in q.__all__ and b in q.__all__


@pytest.mark.parametrize("name", NAMES)
def test_the_other_cache_is_refused(q, name):  # noqa: F811
    other = NAMES[NAMES.index(name) ^ 1]
    with pytest.raises(ValueError, match="the call takes a cache of"):
        getattr(q, name)(*args_of(q, other))
