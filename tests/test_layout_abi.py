"""The binding and the library agree on the structs that calls pass, or the binding says so."""
import ctypes

import pytest

from varlen_gqa_attention_paged_gb300 import _lib


def test_the_library_tells_the_size_of_its_shape_struct():
    assert _lib.load().ua_shape_bytes() == ctypes.sizeof(_lib.UaShape)


class _Library:
    """What the binding sees of a loaded library: ua_shape_bytes, if it has one."""

    def __init__(self, size):
        if size is not None:
            class Size:
                def __call__(self):
                    return size
            self.ua_shape_bytes = Size()


def test_a_library_of_another_header_is_refused():
    _lib._check_layout(_Library(ctypes.sizeof(_lib.UaShape)))
    for size in (None, ctypes.sizeof(_lib.UaShape) - 48):
        with pytest.raises(RuntimeError, match="another version"):
            _lib._check_layout(_Library(size))


def test_the_device_check_names_what_raises_it():
    text = _lib.load().ua_status_string(_lib.UA_ERR_DEVICE_CHECK)
    for what in (b"block id", b"position", b"max_seqlen_q"):
        assert what in text
