"""The 4-bit cache's calls without a GPU: sizes that are no numbers of bytes."""
import ctypes

import pytest

from coalesced_packed_attention_gb300 import zl
from tests._lib import ensure_library


@pytest.fixture(scope="module", autouse=True)
def lib():
    return ensure_library()


def test_a_workspace_past_63_bits_is_refused(lib):
    b = ctypes.c_int64(-1)
    c = zl.zl_kv4_cache(1 << 20, 1024, 64, 256, 1 << 16, 9, 0x1000, 0x2000, 0x3000, 0x4000)
    assert lib.zl_kv4_attn_workspace(c, 1024, 8192, 1, ctypes.byref(b)) == zl.ZL_ERR_UNSUPPORTED and b.value == -1
    assert lib.zl_kv4_attn_workspace(c, 1024, 8192, 0, ctypes.byref(b)) == zl.ZL_OK and 0 < b.value < 1 << 30
    assert lib.zl_kv4_attn_workspace(c, 1024, 8, 1, ctypes.byref(b)) == zl.ZL_OK and b.value > (1 << 20) * 1024 * (1 << 24) * 8 * 4
    assert lib.zl_kv4_evict_workspace(c, ctypes.byref(b)) == zl.ZL_OK and b.value >= (1 << 20) * 1024 * (1 << 24) * 8


def test_no_tokens_have_no_positions(lib):
    c = zl.zl_kv4_cache(2, 2, 64, 16, 4, 9, 0x1000, 0x2000, 0x3000, 0x4000)
    assert lib.zl_kv4_write(c, None, 128, None, 128, 0, 0x30000, None, 0x50000, None) == zl.ZL_OK
    assert lib.zl_kv4_write(c, 0x10000, 128, 0x20000, 128, 1, 0x30000, None, 0x50000, None) == zl.ZL_ERR_INVALID_ARG
