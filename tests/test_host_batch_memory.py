"""The batch builder refuses results that share memory with the lengths it reads."""
import ctypes

import pytest

import __graft_entry__

AT, FAR, B = 1 << 20, 1 << 24, 100  # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def api():
    __graft_entry__.build()
    from deepseek_sparse_attention_fp8_gb300 import api as a

    return a


@pytest.mark.parametrize("name", ["seq", "qsl"])
@pytest.mark.parametrize("lengths", ["ctx", "new"])
@pytest.mark.parametrize("off", [-4 * B + 4, -4, 0, 4, 4 * B - 4])
def test_overlap(api, name, lengths, off):
    at = dict(ctx=FAR, new=FAR + (1 << 16), seq=FAR + (2 << 16), qsl=FAR + (3 << 16))
    at[lengths], at[name] = AT, AT + off
    p = {k: ctypes.c_void_p(v) for k, v in at.items()}
    rest = [ctypes.c_void_p(FAR + (i << 16)) for i in range(4, 8)]
    st = api.lib.dsa_build_batch(p["ctx"], p["new"], B, 64, None, 0, None, None, rest[0], 4, 8, p["seq"], p["qsl"],
                                 rest[1], rest[2], rest[3], None, None)
    assert st == api.DSA_ERR_INVALID_ARG and b"memory" in api.lib.dsa_last_error()
