"""Uses of the prompt path that can be checked without a GPU: one token in place, rows of a wider tensor."""
import ctypes

import pytest
import torch

FAKE = ctypes.c_void_p(0x10000)      # never dereferenced: without a GPU the call ends at the device check
INVALID_ARG = 1


@pytest.fixture(scope="module")
def lib():
    from quantized_speculative_decoding_packed_b200 import build
    build.build()
    from quantized_speculative_decoding_packed_b200 import qspec
    return qspec


def _turn_in_place(lib, tokens, ld_qkv, ld_q):
    return lib.LIB.qspec_qkv_rope_append(FAKE, ld_qkv, tokens, 1, None, 4, 2, 128, None, None, 1e-6, None, 0, 0, None,
                                         ctypes.c_void_p(0x8000), 0, ctypes.c_void_p(0x1000000), ctypes.c_void_p(0x2000000),
                                         8, FAKE, ld_q, lib.ROPE_Q_FP32, None, 0, None)


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are not real")
def test_one_token_is_turned_in_place_whatever_the_strides(lib):
    """The stride of a single row says nothing: queries over the projection's own are accepted."""
    assert _turn_in_place(lib, 1, 1024, 512) != INVALID_ARG
    assert _turn_in_place(lib, 1, 1024, 1024) != INVALID_ARG
    assert _turn_in_place(lib, 2, 1024, 1024) != INVALID_ARG
    assert _turn_in_place(lib, 2, 1024, 512) == INVALID_ARG


def test_row_strides_of_the_binding(lib):
    """(address, stride) of rows: those of a slice; one row has the width that is asked for."""
    wide = torch.zeros(3, 1037)
    rows = lambda t, n, c: lib._rows(t, torch.float32, -1, n, c, "x")      # noqa: E731
    assert rows(wide[:, :512], 3, 512) == (wide.data_ptr(), 1037)
    assert rows(wide, 3, 512) == (wide.data_ptr(), 1037)
    assert rows(wide[1:2, 5:517], 1, 512) == (wide[1:2, 5:517].data_ptr(), 512)
    assert rows(wide[1:2], 1, 512) == (wide[1:2].data_ptr(), 512)
    assert rows(wide[:1].expand(3, 1037)[:1], 1, 512) == (wide.data_ptr(), 512)
    with pytest.raises(ValueError):
        rows(wide[:, ::2], 3, 512)


def test_test_hook_of_the_attention_calls(lib):
    """The hook's bit belongs to the two attention calls; what these refuse, they refuse with it."""
    bad = [0x10000, 512, 6, 2, 0x10000, 4, 2, 64, 0x10000, 0x10000, 0x10000, 8, 0x10000000000, 512, 0x10000, 1 << 40]
    call = lambda op, n: lib.LIB.qspec_call(op, lib._PREFILL_ARGS.pack(*bad), n, None)      # noqa: E731
    for op, n in ((1, 16), (0x101, 16), (0x101, 15), (0x100, 16), (0x103, 16), (0x201, 16), (-0xff, 16)):
        assert call(op, n) == INVALID_ARG
