"""The weights of cached keys on streams of their own. The weights' copy is made on the
current stream, which the other stream waits for: nothing else puts the two in order."""
import pytest
import torch

from cache_common import PAGE
from gpu_common import need_gpu
from test_gpu_cache_fwd import make
from test_gpu_cache_weights import forward, ints


@pytest.mark.gpu
@pytest.mark.parametrize("N", [1, 30])
def test_weights_on_another_stream(N):
    fm = need_gpu()
    H, Hk, d, lens = 8, 2, 128, [700, 1300]
    q, cache, table, _ = make(fm, 2, H, Hk, N, d, lens)
    lse = forward(fm, q, cache, table, lens, None, None)
    ln, w0 = ints(lens), torch.rand((cache.k8.shape[0], Hk, PAGE), device="cuda")
    new_ws = lambda: fm.alloc_cache_weights_workspace(2, H, Hk, N, d, table.shape[1])
    call = lambda w, ws, **kw: fm.flashmask_cache_weights(q, cache, table, ln, lse, w, ws, **kw)
    want = call(w0.clone(), new_ws())
    streams = [torch.cuda.Stream() for _ in range(3)]
    held = [(w0.clone(), new_ws()) for _ in streams]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [call(w, ws, stream=s) for s, (w, ws) in zip(streams, held)]
    for s in streams:
        torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(x, want) for x in got)
    assert all(fm.flashmask_check_status(ws) == (fm.FM_OK, 0) for _, ws in held)
