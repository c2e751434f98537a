"""CPU checks of sizes around the multi-head scan: long sequences that a launch cannot cut into chunks,
and calls without heads or channels (no compute call is made; the addresses are never dereferenced)."""
import os

import pytest

from selective_state_space_36_amd import ops
from tests.test_abi_block import call
from tests.test_abi_head import BAD, BWD


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(ops.LIB_PATH):
        from selective_state_space_36_amd import build
        build.build()
    return ops.lib()


@pytest.mark.parametrize("dtype", [ops.SS_F32, ops.SS_BF16])
@pytest.mark.parametrize("heads,P,N", [(48, 16, 16), (48, 64, 64), (6, 512, 16), (1, 64, 128)])
def test_long_walks_are_not_refused(lib, dtype, heads, P, N):
    """Few walks are cut into their chunks, a workgroup each, as long as a launch has so many
    (2^32 - 1 threads, 512 a workgroup); beyond, the call goes on as far as its arguments' check."""
    walks = 2 * heads * ((P + 63) // 64)
    most = (2 ** 32 - 1) // 512 // walks
    for chunks in (most, most + 1, 4 * most, (2 ** 31 - 1) // 64):
        # (chunks of the last launch, one workgroup each and run of heads)
        if chunks * -(-256 // chunks) > (2 ** 32 - 1) // 512:
            continue
        kw = dict(batch=1, H=heads, P=P, N=N, Gr=1, L=64 * chunks, dtype=dtype, x=None)
        assert call(lib, "ss_scan2_bwd", BWD, **kw) == BAD
        assert lib.ss_last_error() == b"x is NULL", chunks
        # states and adjoints of every chunk, and the decays where walks are cut
        need = lib.ss_scan2_bwd_workspace_bytes(1, 64 * chunks, heads, P, 1, N, dtype)
        states = 2 * 4 * chunks * heads * P * N
        assert states <= need <= states + 4 * chunks * heads * 5 + 64
