"""What the embedding's gradient refuses before anything is launched (CPU only)."""
import ctypes

import pytest

import deterministic_attn_backward_gb300 as dab

BF16, I32, I64 = 0, 2, 3


@pytest.fixture(scope="module")
def lib():
    from deterministic_attn_backward_gb300 import build
    build.build()
    return dab.load_library()


@pytest.mark.parametrize("n", [1, 2048, 2049, 100_000])     # one launch, and several
@pytest.mark.parametrize("accumulate", [0, 1])
def test_tokens_are_checked_when_rows_have_no_width(lib, n, accumulate):
    """The kernels read the tokens whatever the width (to report those outside the
    table): a null or misaligned address is refused on the host."""
    ok, none, big = ctypes.c_void_p(32), None, 1 << 40

    def call(ids, wide):
        return lib.dab_embed_bwd(ids, wide, none, BF16, none, BF16, n, 10, 0, 1.0, -1, accumulate, ok, big, None)

    for wide in (I32, I64):
        assert call(none, wide) == 1
        assert call(ctypes.c_void_p(34), wide) == 1
    assert call(ctypes.c_void_p(36), I64) == 1      # aligned to 4 only
