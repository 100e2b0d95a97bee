"""Captured calls of the attention over a cache whose kernels follow one another as dependent
launches (tiles, rows, the joining of their partial results): every replay follows the device's
lengths, token rows and tables, gives the bits of a plain call on the same values, and graphs
with workspaces of their own run beside one another.  And the same bits on every call."""
import pytest
import torch

import _kv_ref as ref
from test_kv_gpu import DEV, Batch, i32, randn

pytestmark = pytest.mark.gpu

CHAINS = [  # n, lens, page, hq, hkv, d, prefix; then what the next replays find: (n, lens)
    (([1] * 20, [500 + 9 * i for i in range(20)], 16, 8, 2, 128, 0),                   # rows
     [([1] * 20, [1 + 33 * i for i in range(20)]), ([0, 1] * 10, [0, 600] * 10)]),
    (([1, 1], [12000, 9000], 64, 3, 1, 128, 0),                    # rows, eight warps join a row
     [([1, 1], [1, 12000]), ([1, 0], [7777, 3])]),
    (([2] * 24, [100 + i for i in range(24)], 16, 8, 2, 64, 5000),                     # tiles, rows
     [([1, 2] * 12, [2 + 4 * i for i in range(24)]), ([0, 2] * 12, [0, 90] * 12)]),
    (([130, 140], [2000, 150], 16, 8, 2, 128, 0),                                      # tiles
     [([140, 1], [150, 1999]), ([0, 100], [0, 1000])]),
    (([1] * 10 + [150] + [1] * 3, [300] * 10 + [400] + [70] * 3, 16, 8, 2, 128, 0),    # mixed
     [([150] + [1] * 13, [150] + [33 * i for i in range(13)]),
      ([1, 2, 4, 5, 60] + [0, 1, 1] * 3, [1, 2, 4, 300, 60] + [0, 390, 1] * 3)]),
    (([1] * 10 + [150] + [1] * 3, [300] * 10 + [400] + [70] * 3, 32, 8, 2, 64, 700),   # all three
     [([150] + [1] * 13, [150] + [33 * i for i in range(13)]),
      ([1, 2, 4, 5, 60] + [0, 1, 1] * 3, [1, 2, 4, 300, 60] + [0, 390, 1] * 3)]),
    (([1] * 10 + [50] + [1] * 3, [300] * 10 + [400] + [70] * 3, 24, 8, 2, 64, 70),     # odd pages
     [([50] + [1] * 13, [50] + [30 * i for i in range(13)])]),
]


def state(x, n, lens):
    """Sizes of a replay in the batch x was made for: cu and lens."""
    return i32([sum(n[:i]) for i in range(len(n) + 1)]), i32(lens)


def capacity(case):
    (n, lens, *rest), replays = CHAINS[case]
    most = [max(c) for c in zip(lens, *(r[1] for r in replays))]
    return n, most, rest, [(n, lens)] + replays


@pytest.mark.parametrize("case", range(len(CHAINS)))
def test_replays_follow_the_device(ra_lib, case):
    n0, most, (page, hq, hkv, d, plen), replays = capacity(case)
    x = Batch(n0, most, page, hkv, d, plen, seed=case, fill=0.0)
    N = max(sum(n) for n, _ in replays)
    kp, vp, tables, pt = x.gpu("kp", "vp", "tables", "ptable")
    cu, lens = (t.to(DEV) for t in state(x, *replays[0]))
    q = randn(N, hq, d, seed=50 + case)
    qs = [q.to(DEV), q.flip(0).to(DEV)]
    bound = max(max(n) for n, _ in replays)
    kw = dict(max_len=max(most), prefix_table=pt, prefix_len=plen)

    def call(i, **more):
        return ra_lib.prefix_attn_fwd(qs[i], kp, vp, cu, lens, tables, bound, **kw, **more)

    call(0)
    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            res = call(i)
        graphs.append((g, res))
    side = torch.cuda.Stream()
    for n, ln in replays + replays[:1]:
        c, l = state(x, n, ln)
        cu.copy_(c)
        lens.copy_(l)
        for _, (o, s) in graphs:
            o.fill_(7.0)
            s.fill_(7.0)
        torch.cuda.synchronize()
        for _ in range(2):  # one after another, and the two beside one another
            graphs[0][0].replay()
            with torch.cuda.stream(side):
                graphs[1][0].replay()
        torch.cuda.synchronize()
        rows = sum(n)
        for i, (_, (o, s)) in enumerate(graphs):
            plain = call(i, out=torch.full_like(o, 7.0), lse=torch.full_like(s, 7.0))
            assert ra_lib.ra_sync_status() == 0
            assert torch.equal(o, plain[0]) and torch.equal(s, plain[1]), (n, ln)
            assert (o[rows:] == 7).all() and (s[:, rows:] == 7).all()
            want = ref.prefix_attention(qs[i][:rows].cpu(), x.kp, x.vp, c, l, x.tables, x.ptable,
                                        plen, d ** -0.5)
            ref.check_attention(o[:rows], s[:, :rows].t(), (want[0], want[1], want[2].t()),
                                f"{n} {ln}")


@pytest.mark.parametrize("case", range(len(CHAINS)))
def test_same_bits_on_every_call(ra_lib, case):
    n, most, (page, hq, hkv, d, plen), _ = capacity(case)
    x = Batch(n, most, page, hkv, d, plen, seed=case)
    args = (randn(x.N, hq, d, seed=case).to(DEV), *x.gpu("kp", "vp", "cu", "lens", "tables"),
            max(n))
    kw = dict(max_len=max(most), prefix_table=x.ptable.to(DEV), prefix_len=plen)
    first = [t.clone() for t in ra_lib.prefix_attn_fwd(*args, **kw)]
    for _ in range(20):
        o, l = ra_lib.prefix_attn_fwd(*args, **kw)
        assert torch.equal(o, first[0]) and torch.equal(l, first[1])


def test_captured_decoder_step(ra_lib):
    """Append, then attention that reads what it wrote, in one graph: each replay writes and reads
    at the lengths that it finds."""
    hq, hkv, d, page, plen, B = 8, 2, 128, 16, 3000, 24
    x = Batch([1] * B, [200] * B, page, hkv, d, plen, seed=1, fill=0.0)
    kp, vp, cu, lens, tables, pt = x.gpu("kp", "vp", "cu", "lens", "tables", "ptable")
    qkv = randn(B, hq + 2 * hkv, d, seed=2).to(DEV)
    inv = (10000.0 ** (-torch.arange(0, d, 2) / d)).float()
    dinv = inv.to(DEV)

    def step():
        q = ra_lib.paged_kv_append(qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], kp, vp, cu,
                                   lens, tables, dinv, 1, pos_offset=plen)
        return q, *ra_lib.prefix_attn_fwd(q, kp, vp, cu, lens, tables, 1, max_len=200,
                                          prefix_table=pt, prefix_len=plen)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q, o, l = step()
    for at in range(3):
        now = i32([1 + (60 * at + 17 * b) % 200 for b in range(B)])
        lens.copy_(now)
        qkv.copy_(randn(B, hq + 2 * hkv, d, seed=3 + at))
        graph.replay()
        assert ra_lib.ra_sync_status() == 0
        k, v = kp.cpu(), vp.cpu()
        for b in range(B):
            place = int(x.tables[b, (int(now[b]) - 1) // page]), (int(now[b]) - 1) % page
            assert torch.equal(v[place], qkv[b, hq + hkv:].cpu())
        want = ref.prefix_attention(q.cpu(), k, v, x.cu, now, x.tables, x.ptable, plen, d ** -0.5)
        ref.check_attention(o, l.t(), (want[0], want[1], want[2].t()), f"replay {at}")
