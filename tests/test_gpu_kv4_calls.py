"""The 4-bit cache on the GPU: calls that the documentation allows, one after another, at once and with state that goes on."""
import numpy as np
import pytest

from coalesced_packed_attention_gb300 import zl
from oracle import kv4 as ref
from tests._lib import ensure_library
from tests.test_gpu_kv4 import F, f64, make_cache, many, reference, run_attention, starts_of, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    return ensure_library()


@pytest.mark.parametrize("d,page,lens,weights", [(128, 16, [33, 500, 1, 130], False), (64, 64, [200] * 24, True), (128, 256, [250] * 200, False)])
def test_short_calls_one_after_another(d, page, lens, weights):
    """Clusters of every size, launch behind launch, each with outputs of its own: every one of them the first one's."""
    import torch
    c, data, pages = make_cache(lens, 2, d, page, 70)
    n, times = len(lens), 200
    want = run_attention(c, data, pages, lens, [1] * n, 4, 71, no_starts=True)
    q = torch.randn(n, 8, d, generator=torch.Generator().manual_seed(71)).bfloat16().cuda()[:, 4:]
    o, lse = torch.full((times, n, 4, d), 7.0, dtype=torch.bfloat16).cuda(), torch.full((times, n, 4), 7.0).cuda()
    w = torch.zeros((times, *c.slot_shape)).cuda() if weights else [None] * times
    ws = torch.empty(zl.zl_kv4_attn_workspace_bytes(c, 4, 1, weights), dtype=torch.uint8).cuda()
    for i in range(times):
        zl.zl_kv4_attn_fwd(c, q, o[i], lse[i], ws, d ** -0.5, weights_out=w[i])
    assert zl.zl_kv4_get_device_status(c) == 0
    first = (o[0], lse[0]) if weights else want
    assert all(torch.equal(x, first[0]) for x in o) and all(torch.equal(x, first[1]) for x in lse)
    assert not weights or all(torch.equal(x, w[0]) for x in w)
