"""Calls of the paged 4-bit cache at the edges of what their documentation allows."""
import ctypes
import threading

import numpy as np
import pytest
import torch

from oracle import paged
from tests.test_paged_gpu import THETA, _check, _cuda, _pool, _rope, _tables

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


@pytest.mark.parametrize("D,n_q,n_kv", [(128, 8, 2), (64, 16, 2)])
@pytest.mark.parametrize("scale,qscale", [(1.0, 1e4), (1.0, 1e5), (1.0, 1e6), (1.0, 1e7), (1.0, 1e12), (1.0, 1e33), (1e-3, 1e40),
                                          (300.0, 1e3)])
def test_large_scores(dl, D, n_q, n_kv, scale, qscale):
    """Scores up to f32's range.  Each query is a key of its sequence times `qscale`, which beats every other key by far
    more than a score's error, so that the weights are 1 and 0; in the second sequence all pages hold the same keys and
    values of their own, whose scores are equal bit for bit.  The bound is the attention's without the error of scores."""
    rng = np.random.default_rng(int(np.log10(qscale)) + D)
    page, lens, G = 32, [3000, 40 * 32, 1, 40], n_q // n_kv
    tables, n_pages = _tables(rng, lens, page)
    pool, _ = _pool(rng, n_pages, n_kv, page, D, scale)
    pool[tables[1, 1:40], ..., :9 * D] = pool[tables[1, 0], ..., :9 * D]
    K, V = paged.keys_values(pool, D)
    q = np.zeros((4, n_q, D), np.float32)
    for s, n in enumerate(lens):
        for h in range(n_q):
            t = int(rng.integers(0, n))
            q[s, h] = K[tables[s, t // page], h // G, t % page] * qscale
    assert np.isfinite(q).all()
    kw = dict(n_q=n_q, n_kv=n_kv, D=D, page=page)
    q = q.reshape(4, -1)
    lbound = paged.attention(q, pool, tables, lens, **kw)[3]        # (2^-21 (1 + |lse|) and a score's error)
    out, bound, lse = np.zeros((4, n_q, D)), np.zeros((4, n_q, D)), np.zeros((4, n_q))
    for s, n in enumerate(lens):
        for h in range(n_q):
            at = np.arange(n)
            k, v = (x[tables[s, at // page], h // G, at % page] for x in (K, V))
            sc = (k * q[s].reshape(n_q, D)[h].astype(np.float64)).sum(-1) / np.sqrt(D)
            top = (k == k[sc.argmax()]).all(-1)
            if not top.all():
                assert (sc.max() - sc[~top]).min() > 2 * lbound[s, h] + 100
            out[s, h], lse[s, h] = v[top].mean(0), sc.max() + np.log(top.sum())
            bound[s, h] = (2.0 ** -19 + n / 16 * 2.0 ** -23) * np.abs(v[top]).mean(0) + \
                (n * 2.0 ** -32 + 2.0 ** -29) * np.abs(v).max()
    gp, gq, gt, gl = _cuda(pool, q, tables, np.array(lens, np.int32))
    ls = torch.empty(4, n_q, device="cuda")
    got = dl.dl_paged_attn(gq, dl.PagedKV(gp, page, D), gt, gl, dl.paged_attn_workspace(n_q, n_kv, D), n_q, None, ls)
    _check(got.cpu().numpy(), ls.cpu().numpy(), (out.reshape(4, -1), lse, bound.reshape(4, -1), lbound))


def test_select_from_two_threads(dl):
    """Tables of different widths, each past the default limit of shared memory, from two host threads at once (the C
    calls, which ctypes makes without the interpreter's lock)."""
    D, page, n_kv, n_q = 64, 16, 1, 4
    rng = np.random.default_rng(3)
    runs = []
    for width in (16384, 5000):                         # the most there may be, and a few more than 4096
        mean = rng.standard_normal((64, n_kv, D)).astype(np.float16)
        tables = rng.integers(0, 64, (1, width)).astype(np.int32)
        q = rng.standard_normal((1, n_q * D)).astype(np.float32)
        lens = [width * page]
        want = paged.select(q, mean, tables, lens, n_q=n_q, n_kv=n_kv, D=D, page=page, top_k=5, sink=1, local=2)
        gm, gt, gq, gl = _cuda(mean, tables, q, np.array(lens, np.int32))
        kv = dl.PagedKV(dl.PagedKV.empty(64, n_kv, page, D).pool, page, D, k_mean=gm)
        pages, stream = torch.zeros(1, n_kv, 8, dtype=torch.int32, device="cuda"), torch.cuda.Stream()
        c = dl.dl_block_tables(gt.data_ptr(), width, 1, width)
        ptr = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
        args = (ptr(gq), n_q * D, ctypes.byref(kv.c), ctypes.byref(c), ptr(gl), 1, n_q, 5, 1, 2, ptr(pages), None,
                ctypes.c_void_p(stream.cuda_stream))
        runs.append((args, pages, want, (gm, gt, gq, gl, kv, c, stream)))
    torch.cuda.synchronize()
    refused, ready = [], threading.Barrier(2)

    def work(args):
        ready.wait(timeout=60)
        refused.append(sum(dl.lib().dl_paged_select(*args) != dl.DL_OK for _ in range(3000)))

    threads = [threading.Thread(target=work, args=r[:1]) for r in runs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert refused == [0, 0]
    for _, pages, want, _ in runs:
        assert np.array_equal(pages.cpu().numpy(), want)


def test_one_workspace_for_all_calls(dl):
    """Calls of single tokens and of several rows, with heads of 64 and of 128, take turns on one workspace; parts joined
    in groups among them.  Each gives what it gives on a workspace of its own, and leaves the counters zero."""
    rng = np.random.default_rng(14)
    page, n_kv, lens = 16, 2, [5000, 40, 9000]
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    calls = []
    for D, n_q, rows in ((64, 8, 1), (64, 8, 3), (128, 8, 1), (128, 16, 3), (64, 16, 1)):
        tables, n_pages = _tables(rng, lens, page)
        kv = dl.PagedKV.empty(n_pages, n_kv, page, D)
        n = sum(lens)
        seq = np.repeat(np.arange(3), lens).astype(np.int32)
        pos = np.concatenate([np.arange(x) for x in lens]).astype(np.int32)
        gt, gs, gpos, gl = _cuda(tables, seq, pos, np.array(lens, np.int32))
        x = torch.randn(n, n_kv * D, device="cuda")
        dl.dl_paged_append(torch.zeros(n, n_kv * D, device="cuda"), x, x, gpos, gt, _rope(dl, 0, 9000, True), kv, n_kv,
                           row_seq=gs)
        q = torch.randn(3 * rows, n_q * D, device="cuda")
        begin = None if rows == 1 else torch.arange(0, 3 * rows + 1, rows, dtype=torch.int32, device="cuda")
        kw = dict(q=q, kv=kv, tables=gt, seqlen=gl, n_q=n_q, row_begin=begin, max_rows=rows)
        calls.append((kw, dl.dl_paged_attn(workspace=dl.paged_attn_workspace(n_q, n_kv, D), **kw)))
    ws = dl.paged_attn_workspace(16, n_kv, 128)
    for i in [0, 1, 0, 2, 0, 3, 4, 1, 4, 2, 1, 3, 2, 0]:
        kw, want = calls[i]
        assert torch.equal(dl.dl_paged_attn(workspace=ws, **kw), want), i
        assert (ws[:48 * sms] == 0).all()               # three counters for each of up to four CTAs an SM


def test_empty_batches(dl):
    """Steps of no rows, from tensors without elements (whose address is 0), leave everything as it was."""
    D, page, n_q, n_kv = 64, 16, 4, 2
    kv = dl.PagedKV.empty(4, n_kv, page, D, means=True)
    kv.pool.fill_(17)
    kv.k_mean.fill_(3.0)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    f32 = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    ws, rope = dl.paged_attn_workspace(n_q, n_kv, D), dl.make_rope(THETA, D, 32)
    status = i32(1)
    for tables in (i32(0, 3), i32(2, 3)):
        n = tables.shape[0]
        for seq in (None, i32(0)):
            dl.dl_paged_append(f32(0, n_q * D), f32(0, n_kv * D), f32(0, n_kv * D), i32(0), tables, rope, kv, n_q, row_seq=seq,
                               q_out=f32(0, n_q * D), k_out=f32(0, n_kv * D), v_out=f32(0, n_kv * D), status=status)
        out = dl.dl_paged_attn(f32(0, n_q * D), kv, tables, i32(n), ws, n_q, lse=f32(0, n_q), row_begin=i32(n + 1), max_rows=2,
                               status=status)
        assert out.shape == (0, n_q * D)
    none = i32(0, 3)
    assert dl.dl_paged_attn(f32(0, n_q * D), kv, none, i32(0), ws, n_q, status=status).shape == (0, n_q * D)
    pages = dl.dl_paged_select(f32(0, n_q * D), kv, none, i32(0), n_q, top_k=2, n_sink=1, n_local=1, status=status)
    assert pages.shape == (0, n_kv, 4)
    dl.dl_paged_attn(f32(0, n_q * D), kv, none, i32(0), ws, n_q, pages=pages, status=status)
    rows = torch.full((3, n_q * D), 7.0, device="cuda")        # rows of no sequence
    out = rows.clone()
    dl.dl_paged_attn(rows, kv, none, i32(0), ws, n_q, out, row_begin=i32(1), max_rows=2, status=status)
    assert dl.dl_status_read(status) == 0
    assert (out == 7.0).all() and (kv.pool == 17).all() and (kv.k_mean == 3.0).all() and (ws == 0).all()
    # rows whose sequences no table knows are skipped as others outside the tables are
    dl.dl_paged_append(f32(2, n_q * D), f32(2, n_kv * D), f32(2, n_kv * D), i32(2), none, rope, kv, n_q, row_seq=i32(2),
                       status=status)
    assert dl.dl_status_read(status) == dl.DL_STATUS_REGION_RANGE and (kv.pool == 17).all()


def test_empty_page_list(dl):
    """A list without room for a page is refused (its tensor has no address, which would read every page)."""
    D, page, n_q, n_kv = 64, 16, 4, 2
    kv = dl.PagedKV.empty(4, n_kv, page, D)
    kv.pool.zero_()
    q = torch.zeros(2, n_q * D, device="cuda")
    tables, lens = torch.zeros(2, 3, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        dl.dl_paged_attn(q, kv, tables, lens, dl.paged_attn_workspace(n_q, n_kv, D), n_q,
                         pages=torch.zeros(2, n_kv, 0, dtype=torch.int32, device="cuda"))


def test_results_made_on_the_named_stream(dl):
    """A result that the call makes itself is memory of the stream it runs on: not a block that the current stream's
    queued work still reads."""
    D, page, n_q, n_kv, n = 64, 16, 8, 2, 64
    rng = np.random.default_rng(4)
    tables, n_pages = _tables(rng, [page] * n, page)
    pool, mean = _pool(rng, n_pages, n_kv, page, D)
    gp, gm, gt = _cuda(pool, mean, tables)
    kv = dl.PagedKV(gp, page, D, k_mean=gm)
    q, lens = torch.ones(n, n_q * D, device="cuda"), torch.full((n,), page, dtype=torch.int32, device="cuda")
    ws, side = dl.paged_attn_workspace(n_q, n_kv, D), torch.cuda.Stream()
    big = torch.zeros(1 << 28, device="cuda")
    kw = dict(top_k=61, n_sink=1, n_local=2)
    calls = (((n, n_q * D), torch.float32, lambda: dl.dl_paged_attn(q, kv, gt, lens, ws, n_q, stream=side)),
             ((n, n_kv, 64), torch.int32, lambda: dl.dl_paged_select(q, kv, gt, lens, n_q, stream=side, **kw)))
    for shape, dtype, call in calls:
        call()                                          # (first launches load code)
        kept = torch.full(shape, 7, dtype=dtype, device="cuda")
        seen = torch.zeros_like(kept)
        torch.cuda.synchronize()
        for _ in range(20):                             # some milliseconds before the read
            big.add_(1.0)
        seen.copy_(kept)
        del kept
        got = call()
        torch.cuda.synchronize()
        assert (seen == 7).all()
        assert got.shape == shape


@pytest.mark.parametrize("n", [48, 700])
@pytest.mark.parametrize("with_seq", [True, False])
def test_append_arguments_of_the_kernel_before(dl, n, with_seq):
    """Positions, sequences and table entries that the kernel right before the store writes (another store, whose q
    without rotation carries their bits): the store's two launches must go by them, not by what was there."""
    D, page, n_kv, cols = 64, 16, 2, 64
    rng = np.random.default_rng(n)
    if with_seq:                                        # prompts of a few sequences, pages filled throughout
        lens = [n - n // 3, n // 3]
        seq, pos = np.repeat(np.arange(2), lens), np.concatenate([np.arange(x) for x in lens])
    else:                                               # a row each, half of them filling a page
        lens = [int(x) for x in rng.integers(1, 60, n)]
        lens[::2] = [page * int(x) for x in rng.integers(1, 4, len(lens[::2]))]
        seq, pos = np.arange(n), np.array(lens) - 1
    tables, n_pages = _tables(rng, lens, page, width=64)
    pool, mean = _pool(rng, n_pages, n_kv, page, D)
    k, v = (rng.standard_normal((n, n_kv * D)).astype(np.float32) for _ in range(2))
    wide = lambda x: np.concatenate([x, np.zeros(-len(x) % cols, x.dtype)]).reshape(-1, cols).astype(np.int32)  # noqa: E731
    good = dict(pos=wide(pos), seq=wide(seq), tab=tables)
    bad = dict(pos=wide(rng.choice([-1, page - 1, 1 << 30, 0], n)), seq=wide(rng.choice([-1, 1, 1 << 30, 0], n)),
               tab=rng.choice([-1, n_pages, 0, 1 << 30], tables.shape).astype(np.int32))
    # padding where every other argument is still the old one: an early look must not be followed
    put_src = {(w, i): torch.from_numpy(x[w]).cuda().view(torch.float32) for i, x in enumerate((good, bad)) for w in x}
    words = {w: torch.zeros_like(put_src[w, 0]) for w in good}
    m = max(len(x) for x in words.values())
    other = dl.PagedKV.empty(m, 1, page, D)
    own, zero = torch.arange(m, dtype=torch.int32, device="cuda").view(m, 1), torch.zeros(m, dtype=torch.int32, device="cuda")
    kvx, rope = torch.zeros(m, D, device="cuda"), _rope(dl, 0, 4096, False)

    def put(what, i):
        x = put_src[what, i]
        c = len(x)
        dl.dl_paged_append(x, kvx[:c], kvx[:c], zero[:c], own[:c], rope, other, 1, q_out=words[what])

    order = ["pos", "seq", "tab"] if with_seq else ["pos", "tab"]
    caches = []
    for _ in order:
        gp, gm = _cuda(pool, mean)
        caches.append(dl.PagedKV(gp, page, D, k_mean=gm))
    gk, gv = _cuda(k, v)
    gq, status = torch.zeros(n, D * n_kv, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    args = {w: words[w].view(torch.int32) for w in words}

    def run():
        for last, kv in zip(order, caches):
            for w in order:
                put(w, w == last)
            put(last, 0)                                # the kernel right before the store
            dl.dl_paged_append(gq, gk, gv, args["pos"].view(-1)[:n], args["tab"], rope, kv, n_kv,
                               row_seq=args["seq"].view(-1)[:n] if with_seq else None, status=status)

    want_pool, want_mean = pool.copy(), mean.copy()
    paged.append(want_pool, want_mean, np.zeros((n, n_kv * D), np.float32), k, v, pos, seq, tables, n_q=n_kv, n_kv=n_kv, D=D,
                 page=page, rot=0, theta=THETA, neox=False)

    def check():
        torch.cuda.synchronize()
        assert dl.dl_status_read(status) == 0
        for kv in caches:
            assert np.array_equal(kv.pool.cpu().numpy(), want_pool) and np.array_equal(kv.k_mean.cpu().numpy(), want_mean)
            kv.pool.copy_(torch.from_numpy(pool))
            kv.k_mean.copy_(torch.from_numpy(mean))

    run()
    check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for _ in range(3):
        g.replay()
        check()


@pytest.mark.parametrize("qscale", [1e10, 1e20, 1e30, 1e36, 6e37])
@pytest.mark.parametrize("D,n_q,n_kv", [(128, 16, 2), (64, 6, 3)])
def test_select_large_queries(dl, D, n_q, n_kv, qscale):
    """Finite queries whose sums, products or scores pass f32 on the way are ranked as 64 bits rounded to f32 rank them:
    scores past f32 are infinite and tie, the others count; pages of zeros and of small means are among them."""
    rng = np.random.default_rng(int(np.log10(qscale)))
    page, n = 16, 1500
    lens, tables = [n * page] * 2, np.arange(2 * n, dtype=np.int32).reshape(2, n)
    mean = (rng.standard_normal((2 * n, n_kv, D)) * 10.0 ** rng.integers(-4, 2, (2 * n, n_kv, 1))).astype(np.float16)
    mean[rng.integers(0, 2 * n, 60), :, ::2] = 0.0
    mean[rng.integers(0, 2 * n, 60)] = 0.0
    q = (rng.uniform(-5, 5, (2, n_q * D)) * qscale).astype(np.float32)
    q[1, :n_q * D // 2] = np.abs(q[1, :n_q * D // 2])   # the group's sum passes f32 at the largest size
    assert np.isfinite(q).all()
    kw = dict(n_q=n_q, n_kv=n_kv, D=D, page=page, top_k=400, sink=1, local=2)
    want = paged.select(q, mean, tables, lens, **kw)
    gq, gm, gt, gl = _cuda(q, mean, tables, np.array(lens, np.int32))
    kv = dl.PagedKV(dl.PagedKV.empty(2 * n, n_kv, page, D).pool, page, D, k_mean=gm)
    got = dl.dl_paged_select(gq, kv, gt, gl, n_q, top_k=400, n_sink=1, n_local=2)
    assert np.array_equal(got.cpu().numpy(), want)
