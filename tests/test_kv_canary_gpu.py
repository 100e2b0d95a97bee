"""Guard canaries of the cache and cross-attention operators: every output, the cache's pages and
a workspace of exactly the reported bytes lie inside larger buffers whose guard regions must be
unchanged after the call.  Odd numbers of rows, so that every region of the workspace ends off
a 16-byte border; each kernel and each way of joining partial results."""
import pytest
import torch

import _kv_ref as ref
from test_canary_gpu import guarded, intact, written
from test_kv_gpu import DEV, Batch, i32, randn

pytestmark = pytest.mark.gpu

PLANS = [  # n, lens, page, hq, hkv, d, prefix
    ([1, 1, 1], [300, 40, 17], 16, 6, 2, 64, 100),            # clusters
    ([3, 2], [70, 9], 16, 9, 1, 128, 0),
    ([1] * 75, [1 + 13 * i % 900 for i in range(75)], 16, 3, 1, 64, 0),     # rows
    ([1] * 75, [1 + 13 * i % 900 for i in range(75)], 16, 5, 5, 128, 77),
    ([1], [9000], 64, 3, 1, 128, 0),                          # eight warps join a row
    ([3, 4], [5000, 17], 16, 3, 1, 64, 0),
    ([41, 1, 30], [41, 300, 60], 5, 3, 1, 64, 31),            # row tiles counted by token rows
    ([33, 2, 1], [50, 3, 1], 24, 3, 3, 128, 0),
    ([131], [131], 16, 3, 1, 64, 0),                          # tiles, written without partials
    ([131, 60], [900, 60], 16, 3, 1, 128, 0),                 # tiles in ranges of keys
    ([21], [21], 16, 3, 1, 128, 2100),                        # two warpgroups to a row tile
    ([1] * 51, [40 + i for i in range(51)], 16, 5, 1, 128, 3000),           # tiles and rows
    ([1, 1, 1, 100], [50, 300, 1, 100], 16, 7, 1, 128, 0),    # mixed
    ([1, 1, 2, 130], [50, 1300, 2, 777], 16, 3, 3, 64, 500),
    ([1, 0, 1, 31], [50, 0, 700, 33], 16, 49, 1, 64, 0),      # packed tiles alone
]


def workspace(nbytes):
    """A buffer of exactly nbytes between guards, as (whole, view): 16-byte aligned, its end
    wherever it falls."""
    whole = torch.full((nbytes + 8192,), 0xA5, dtype=torch.uint8, device=DEV)
    return whole, whole[4096:4096 + nbytes]


def untouched(whole, nbytes):
    torch.cuda.synchronize()
    return bool((whole[:4096] == 0xA5).all()) and bool((whole[4096 + nbytes:] == 0xA5).all())


@pytest.mark.parametrize("case", range(len(PLANS)))
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_prefix_attention_writes_only_its_outputs(ra_lib, case, dtype):
    n, lens, page, hq, hkv, d, plen = PLANS[case]
    x = Batch(n, lens, page, hkv, d, plen, seed=case)
    q = randn(x.N, hq, d, seed=case)
    need = ra_lib.load().ra_prefix_attn_workspace(len(n), x.N, max(n), max(max(lens), 1), plen, hq,
                                                  hkv, d, page)
    ws, view = workspace(need)
    ob, o = guarded((x.N, hq, d), dtype)
    lb, l = guarded((hq, x.N), torch.float32)
    ra_lib.prefix_attn_fwd(q.to(DEV), *x.gpu("kp", "vp", "cu", "lens", "tables"), max(n),
                           max_len=max(max(lens), 1), prefix_table=x.ptable.to(DEV),
                           prefix_len=plen, out=o, lse=l, workspace=view)
    assert ra_lib.ra_sync_status() == 0
    assert intact(ob, o.numel()) and intact(lb, l.numel()) and untouched(ws, need)
    want = ref.prefix_attention(q, x.kp, x.vp, x.cu, x.lens, x.tables, x.ptable, plen, d ** -0.5)
    ref.check_attention(o, l.t(), (want[0], want[1], want[2].t()), f"case {case}")


@pytest.mark.parametrize("n,lens,page,hq,hkv,d", [
    ([1, 1, 1], [5, 16, 17], 16, 3, 1, 64),
    ([7, 0, 2], [7, 0, 40], 5, 5, 5, 128),
    ([1, 1, 1, 1, 50], [1, 2, 3, 4, 55], 1, 1, 1, 64),      # blocks over the token rows
])
def test_append_writes_only_its_rows(ra_lib, n, lens, page, hq, hkv, d):
    x = Batch(n, lens, page, hkv, d, seed=3, fill=0.0)
    qkv = randn(x.N, hq + 2 * hkv, d, seed=4).to(DEV)
    bufs = [guarded(x.kp.shape, torch.bfloat16), guarded(x.kp.shape, torch.bfloat16),
            guarded((x.N, hq, d), torch.bfloat16)]
    (_, kp), (_, vp), (_, qo) = bufs
    kp.copy_(x.kp)
    vp.copy_(x.vp)
    inv = torch.rand(d // 2).to(DEV)
    ra_lib.paged_kv_append(qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], kp, vp,
                           *x.gpu("cu", "lens", "tables"), inv, max(n), q_out=qo)
    assert ra_lib.ra_sync_status() == 0
    for buf, view in bufs:
        assert intact(buf, view.numel()) and written(view)


@pytest.mark.parametrize("B,Lq,Lk,hq,hkv,d", [
    (1, 1, 33, 3, 1, 64),          # clusters
    (3, 1, 5001, 1, 1, 128),       # rows
    (1, 131, 77, 3, 1, 64),        # tiles
    (3, 45, 1111, 3, 1, 128),      # tiles in ranges of keys
    (1, 31, 1201, 3, 3, 64),
])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("deterministic", [False, True])
def test_cross_attention_writes_only_its_outputs(ra_lib, B, Lq, Lk, hq, hkv, d, dtype,
                                                 deterministic):
    lib, code = ra_lib.load(), ra_lib.RA_BF16 if dtype == torch.bfloat16 else ra_lib.RA_FP32
    q, do = (randn(B, Lq, hq, d, seed=s).to(DEV) for s in (1, 2))
    k, v = (randn(B, Lk, hkv, d, seed=s).to(DEV) for s in (3, 4))
    lens = i32([Lk - 7 * (b % 2) for b in range(B)]).to(DEV)
    need = lib.ra_cross_attn_workspace(B, Lq, Lk, hq, hkv, d)
    ws, view = workspace(need)
    ob, o = guarded(q.shape, dtype)
    lb, l = guarded((B, hq, Lq), torch.float32)
    ra_lib.cross_attn_fwd(q, k, v, lens, out=o, lse=l, workspace=view)
    assert ra_lib.ra_sync_status() == 0
    assert intact(ob, o.numel()) and intact(lb, l.numel()) and untouched(ws, need)
    assert written(o) and written(l)
    out = o.bfloat16()
    need = lib.ra_cross_attn_bwd_workspace(B, Lq, hq, d, code)
    ws, view = workspace(need)
    bufs = [guarded(t.shape, dtype) for t in (q, k, v)]
    ra_lib.ra_set_bwd_deterministic(deterministic)
    try:
        status = lib.ra_cross_attn_bwd(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), lens.data_ptr(), out.data_ptr(),
            l.data_ptr(), do.data_ptr(), B, Lq, Lk, hq, hkv, d, hq * d, Lq * hq * d, hkv * d,
            Lk * hkv * d, d ** -0.5, ra_lib.RA_BF16, code, *(t.data_ptr() for _, t in bufs),
            view.data_ptr(), need, torch.cuda.current_stream().cuda_stream)
    finally:
        ra_lib.ra_set_bwd_deterministic(False)
    assert status == 0 and ra_lib.ra_sync_status() == 0
    assert untouched(ws, need)
    for buf, t in bufs:
        assert intact(buf, t.numel()) and written(t)
