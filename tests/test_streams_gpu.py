"""Results that a call makes itself lie in memory of the stream it runs on: never in a block that queued work of the
current stream still reads."""
import pytest
import torch

import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dl():
    import row_decode_step_gb300 as m
    from row_decode_step_gb300 import _build
    _build.build()
    m.lib()
    return m


def _planes(r):
    return {"PackedQ8": lambda: [r.qs, r.d], "PackedF16W": lambda: [r.w], "Tensor": lambda: [r],
            "tuple": lambda: list(r)}[type(r).__name__]()


@pytest.mark.parametrize("name", ["q8_pack", "f16w_pack", "gemv_q8", "gemv_f16w", "attention"])
def test_results_made_on_the_named_stream(dl, name):
    n_out, n_in, rows, n_q, n_kv, D, n = 256, 2048, 8, 8, 2, 64, 200
    blocks = synth.q8_0_blocks_from_normal(1, "streams", n_out, n_in).cuda()
    w = synth.f16_weights_from_normal(1, "streams/f16", n_out, n_in).cuda()
    x = torch.ones(rows, n_in, device="cuda")
    W8, W16 = dl.dl_q8_pack(blocks, n_out, n_in), dl.dl_f16w_pack(w)
    kv = dl.KVCache(torch.zeros(1, n_kv, n, D, dtype=torch.float16, device="cuda"),
                    torch.zeros(1, n_kv, n, D, dtype=torch.float16, device="cuda"))
    lens = list(range(n - rows + 1, n + 1))
    plan = dl.dl_attn_plan_build(lens, n_q, n_kv, D)
    ws, sl = dl.workspace_for(plan), torch.tensor(lens, dtype=torch.int32, device="cuda")
    q = torch.ones(rows, n_q * D, device="cuda")
    side = torch.cuda.Stream()
    call = {"q8_pack": lambda: dl.dl_q8_pack(blocks, n_out, n_in, stream=side),
            "f16w_pack": lambda: dl.dl_f16w_pack(w, stream=side),
            "gemv_q8": lambda: dl.dl_gemv_q8(W8, x, stream=side),
            "gemv_f16w": lambda: dl.dl_gemv_f16w(W16, x, stream=side),
            "attention": lambda: dl.decode_attention(q, kv, sl, plan, ws, stream=side)}[name]
    sizes = [t.numel() * t.element_size() for t in _planes(call())]     # (first launches load code)
    big = torch.zeros(1 << 28, device="cuda")
    torch.cuda.synchronize()
    kept = [torch.full((b,), 77, dtype=torch.uint8, device="cuda") for b in sizes]
    seen = [torch.zeros_like(t) for t in kept]
    torch.cuda.synchronize()
    for _ in range(20):                                 # some milliseconds before the read
        big.add_(1.0)
    for a, b in zip(seen, kept):
        a.copy_(b)
    kept.clear()
    del b
    got = _planes(call())
    torch.cuda.synchronize()
    assert all((t == 77).all() for t in seen)
    assert [t.numel() * t.element_size() for t in got] == sizes
