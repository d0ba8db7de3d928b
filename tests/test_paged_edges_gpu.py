"""Calls of the paged 4-bit cache at the edges of what their documentation allows."""
import numpy as np
import pytest
import torch

from oracle import paged
from tests.test_paged_gpu import _cuda, _pool, _tables

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dl():
    import row_decode_step_gb300 as m
    from row_decode_step_gb300 import _build
    _build.build()
    m.lib()
    return m


@pytest.mark.parametrize("D,n_q,n_kv", [(64, 6, 2), (128, 4, 1), (64, 16, 2), (128, 16, 2)])
def test_odd_queries_of_cut_items(dl, D, n_q, n_kv):
    """A NaN or infinite query's out and lse are NaN whatever its length: an item that one CTA takes, one of a few
    parts, one whose parts are joined in groups (each CTA takes 16 chunks of 32 keys or more); others are untouched."""
    rng = np.random.default_rng(D + n_q)
    page, lens = 32, [300, 1500, 9000, 9000]
    tables, n_pages = _tables(rng, lens, page)
    pool, _ = _pool(rng, n_pages, n_kv, page, D)
    q = rng.standard_normal((4, n_q * D)).astype(np.float32)
    want = paged.attention(q, pool, tables, lens, n_q=n_q, n_kv=n_kv, D=D, page=page)
    bad = np.zeros((4, n_q), bool)
    for s, (h, x) in enumerate(((1, np.nan), (2, np.nan), (0, np.nan), (3, np.inf))):
        q[s, h * D + 5] = x
        bad[s, h] = True
    gp, gq, gt, gl = _cuda(pool, q, tables, np.array(lens, np.int32))
    lse = torch.empty(4, n_q, device="cuda")
    out = dl.dl_paged_attn(gq, dl.PagedKV(gp, page, D), gt, gl, dl.paged_attn_workspace(n_q, n_kv, D), n_q, None, lse)
    o, ls = out.cpu().numpy().reshape(4, n_q, D), lse.cpu().numpy()
    assert np.isnan(o[bad]).all()
    assert np.isnan(ls[bad]).all(), ls[bad]
    ok = np.abs(o - want[0].reshape(4, n_q, D)) <= want[2].reshape(4, n_q, D)
    assert ok[~bad].all() and (np.abs(ls - want[1]) <= want[3])[~bad].all()
