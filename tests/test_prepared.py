"""Prepared calls convert their arguments once (CPU only: every call here is
refused on the host, or has nothing to do)."""

import ctypes as C

import pytest

from pagedattention_decode_attention_gb300 import build, capi, ops


@pytest.fixture(scope="module")
def lib():
    build.build()
    return capi.lib()


ARGS = (256, 256, 256, 256, 256, 1, 8, 128, 16, 2, None)


def test_the_same_call_without_declared_types(lib):
    fn, args = ops._bound(lib.pa_kv_append, ARGS)
    assert fn.argtypes is None and lib.pa_kv_append.argtypes is not None
    for a, t in zip(args, lib.pa_kv_append.argtypes):
        assert type(a) is t
    for change, status in (({5: 0}, 0), ({0: 8}, 1), ({9: 7}, 2), ({7: 96}, 2), ({5: -1}, 1)):
        given = [change.get(i, a) for i, a in enumerate(ARGS)]
        fn, args = ops._bound(lib.pa_kv_append, given)
        assert fn(*args) == status == lib.pa_kv_append(*given)


def test_pointers_keep_their_64_bits(lib):
    fn, args = ops._bound(lib.pa_kv_append, (1 << 60,) + ARGS[1:])
    assert args[0].value == 1 << 60
    fn, args = ops._bound(lib.pa_rotary, [C.c_void_p(1 << 62)] + [256] * 3 + [64, 0, 1.5, 3, 8, 2, 128]
                          + [1 << 39] * 4 + [2, 512, 512, None])
    assert args[0].value == 1 << 62 and args[6].value == 1.5 and args[11].value == 1 << 39


def test_a_wrong_number_of_arguments_is_refused(lib):
    with pytest.raises(TypeError, match="arguments"):
        ops._bound(lib.pa_kv_append, ARGS[:-1])


def test_errors_are_raised(lib):
    with pytest.raises(capi.PagedAttnError) as e:
        ops.Prepared(lib.pa_kv_append, (8,) + ARGS[1:], ())()
    assert e.value.status == 1 and "aligned" in str(e.value)
    ops.Prepared(lib.pa_kv_append, ARGS[:5] + (0,) + ARGS[6:], ())()
