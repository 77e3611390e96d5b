"""Limits of the operators' C ABI that no call may pass, refused before the device
is touched."""
import ctypes

import pytest

from collective_communication_gb300 import binding as B

S = B.Status
BASE, APART = 1 << 40, 1 << 37  # never dereferenced


@pytest.fixture(scope="module")
def lib():
    from collective_communication_gb300 import build
    build.build()
    return B.load_library()


def test_token_logprobs_refuses_more_tiles_than_it_counts(lib):
    """Rows of several shards make a tile of 1024 columns each; fewer than 2^31 in a call. The last call's size fits, and
    its workspace does not."""
    def call(n, rows, vocab, ws_bytes):
        i64 = ctypes.c_int64 * n
        x = (ctypes.c_void_p * n)(*[BASE + r * APART for r in range(n)])
        out = [BASE + (n + i) * APART for i in range(5)]
        return lib.rar_token_logprobs(x, i64(*[vocab] * n), i64(*[vocab] * n), n, rows, 1, *out[:4], 0, None, None, out[4],
                                      ws_bytes, None)

    for n, rows, vocab in ((8, 1 << 28, 1), (2, 1 << 30, 5), (32, 1 << 25, 1025)):
        assert call(n, rows, vocab, 1 << 30) == S.ERR_ARG
    assert call(8, (1 << 28) - 1, 1, 100) == S.ERR_WORKSPACE
