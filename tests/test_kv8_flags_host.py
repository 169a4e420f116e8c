"""Flags of the attention over the paged 8-bit cache (no GPU)."""

import ctypes

import pytest

from top_sparse_mla_gb300 import native
from top_sparse_mla_gb300.build import build


@pytest.mark.parametrize("flags,good", [(0, True), (native.DSA_KV8_FLAG_TEST_WAIT_TIMEOUT, True), (1, False), (3, False), (4, False),
                                        (1 << 31, False)])
def test_only_the_defined_flags_are_taken(flags, good):
    build()
    lib = native.library()
    p = native.DsaKv8Params()
    assert lib.dsa_kv8_params_init(ctypes.byref(p), 10, 4, 64, 8, 128, 64, 100, 16) == native.DSA_OK
    p.flags = flags
    assert (lib.dsa_kv8_attn_workspace_size(ctypes.byref(p), 152) > 0) == good
