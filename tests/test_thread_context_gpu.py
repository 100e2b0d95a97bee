"""Entry points called on a thread that has made no CUDA call yet (as autograd's backward
thread may not have, when torch's cache serves every allocation): each has to find the
device's context by itself."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu


def on_new_thread(fn):
    got = []

    def body():
        try:
            got.append((True, fn()))
        except Exception as e:  # noqa: BLE001 -- re-raised on the calling thread
            got.append((False, e))

    t = threading.Thread(target=body)
    t.start()
    t.join()
    ok, value = got[0]
    if not ok:
        raise value
    return value


def randn(*shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").bfloat16()


def test_ring_attention_on_a_new_thread(ra_lib):
    q, k, v, do = (randn(*s, seed=i) for i, s in enumerate(
        [(1, 256, 2, 64), (2, 1, 128, 2, 64), (2, 1, 128, 2, 64), (1, 256, 2, 64)]))
    o, l = ra_lib.ring_attn_fwd(q, k, v, True, out_dtype=torch.bfloat16)
    g = ra_lib.ring_attn_bwd(q, k, v, o, l, do, True)
    out, lse = torch.empty_like(o), torch.empty_like(l)
    grads, ws = [torch.empty_like(x) for x in g], torch.empty_like(l)
    s = torch.cuda.current_stream()
    on_new_thread(lambda: ra_lib.ring_attn_fwd(q, k, v, True, out=out, lse=lse, stream=s))
    on_new_thread(lambda: ra_lib.ring_attn_bwd(q, k, v, o, l, do, True, None, *grads, ws,
                                               stream=s))
    torch.cuda.synchronize()
    assert torch.equal(out, o) and torch.equal(lse, l)
    assert torch.equal(grads[1], g[1]) and torch.equal(grads[2], g[2])


def test_cross_attention_on_a_new_thread(ra_lib):
    q, k, v, do = (randn(*s, seed=i) for i, s in enumerate(
        [(2, 130, 4, 64), (2, 70, 2, 64), (2, 70, 2, 64), (2, 130, 4, 64)]))
    o, l = ra_lib.cross_attn_fwd(q, k, v, out_dtype=torch.bfloat16)
    g = ra_lib.cross_attn_bwd(q, k, v, o, l, do)
    want = [x.clone() for x in (o, l, g[1], g[2])]
    for _ in range(2):  # the second round's buffers come from torch's cache
        del o, l, g
        o, l = on_new_thread(lambda: ra_lib.cross_attn_fwd(q, k, v, out_dtype=torch.bfloat16))
        g = on_new_thread(lambda: ra_lib.cross_attn_bwd(q, k, v, o, l, do))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, (o, l, g[1], g[2])))


def test_prefix_attention_on_a_new_thread(ra_lib):
    pages = randn(12, 2, 16, 2, 64, seed=1)
    q = randn(40, 4, 64, seed=2)
    i32 = dict(dtype=torch.int32, device="cuda")
    args = (q, pages[:, 0], pages[:, 1], torch.tensor([0, 40], **i32), torch.tensor([90], **i32),
            torch.arange(6, **i32)[None], 40)
    kw = dict(prefix_table=torch.arange(6, 12, **i32), prefix_len=91)
    want = ra_lib.prefix_attn_fwd(*args, **kw)
    for _ in range(2):
        got = on_new_thread(lambda: ra_lib.prefix_attn_fwd(*args, **kw))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
        del got
