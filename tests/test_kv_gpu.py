"""The operators over a K/V cache on the GPU against plain 64-bit forms: the paged append
with its rotation, attention over the cache behind a shared prefix, the single-token and
short forms of cross attention, and a run of them together."""
import pytest
import torch

import _kv_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
NAN = float("nan")


def randn(*shape, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).bfloat16()


def i32(x):
    return torch.as_tensor(x, dtype=torch.int32)


class Batch:
    """A ragged batch over a paged cache on the CPU: new tokens n[b], own lengths lens[b]."""

    def __init__(self, n, lens, page, hkv, d, plen=0, seed=0, extra_rows=0, spare_pages=3,
                 fill=NAN):
        self.n, self.page = list(n), page
        self.cu = i32([sum(n[:i]) for i in range(len(n) + 1)])
        self.N = int(self.cu[-1]) + extra_rows
        self.lens = i32(lens)
        self.max_pages = max(1, -(-max(list(lens) + [1]) // page))
        n_pre = -(-plen // page)
        used = n_pre + sum(-(-x // page) for x in lens)
        self.n_pages = used + spare_pages
        ids = torch.randperm(self.n_pages, generator=torch.Generator().manual_seed(seed)).tolist()
        self.ptable = i32([ids.pop() for _ in range(n_pre)])
        # entries past a length are not read: an id far outside the cache stands there
        self.tables = torch.full((len(n), self.max_pages), 1 << 29, dtype=torch.int32)
        for b, x in enumerate(lens):
            for j in range(-(-x // page)):
                self.tables[b, j] = ids.pop()
        # rows that hold no key are `fill`
        self.kp = torch.full((self.n_pages, page, hkv, d), fill).bfloat16()
        self.vp = self.kp.clone()
        k, v = randn(used * page, hkv, d, seed=seed + 1), randn(used * page, hkv, d, seed=seed + 2)
        at = 0
        for table, x in [(self.ptable, plen)] + [(self.tables[b], x) for b, x in enumerate(lens)]:
            for j in range(x):
                self.kp[int(table[j // page]), j % page] = k[at]
                self.vp[int(table[j // page]), j % page] = v[at]
                at += 1
        self.plen = plen

    def gpu(self, *names):
        return [getattr(self, n).to(DEV) for n in names]


PREFIX = [  # n, lens, page, hq, hkv, d, prefix
    ([1], [1], 16, 4, 2, 64, 0),
    ([1], [17], 16, 4, 4, 128, 0),
    ([1, 1, 1], [1, 40, 129], 16, 8, 2, 128, 0),
    ([1, 1], [300, 5], 16, 8, 1, 64, 77),
    ([1] * 9, [3, 1, 64, 65, 200, 16, 15, 33, 500], 32, 4, 1, 128, 16),
    ([2, 0, 5, 1], [2, 0, 70, 130], 16, 6, 2, 64, 33),        # a sequence without tokens or keys
    ([3, 1], [10, 2], 5, 4, 2, 64, 12),                       # pages that hold no whole 16 keys
    ([4, 2], [90, 31], 1, 2, 1, 128, 3),                      # one key per page
    ([8, 8, 3], [100, 8, 40], 64, 16, 16, 64, 130),
    ([9, 17], [33, 17], 16, 28, 4, 128, 1),                   # 7 heads per kv head
    ([40, 1, 23], [50, 300, 23], 16, 4, 2, 64, 200),          # several row tiles per sequence
    ([1, 1], [2000, 1], 128, 4, 1, 64, 0),                    # many splits, and one key
    ([2], [2], 256, 8, 8, 128, 3000),
    ([65, 130], [65, 200], 64, 8, 2, 128, 300),
    ([33], [400], 8, 4, 1, 64, 129),
    ([20], [20], 32, 4, 1, 64, 2111),                         # one row tile, odd key tiles
    ([50], [50], 16, 4, 1, 128, 1500),
    ([64, 64], [64, 700], 256, 2, 2, 128, 640),
    ([5, 60], [1, 61], 8, 16, 1, 64, 9),                      # more new tokens than own keys
    ([140], [141], 128, 1, 1, 128, 127),
    ([3, 2], [30, 9], 16, 48, 1, 64, 50),                     # 48 heads per kv head
    ([2, 1], [30, 9], 16, 130, 1, 64, 50),                    # more than a row tile's
    ([5, 3], [40, 100], 16, 4, 1, 64, 0),                     # row tiles of 32
    ([4, 4], [4, 100], 16, 4, 1, 128, 20),
    ([40, 7], [90, 50], 5, 4, 1, 128, 31),                    # many row tiles of odd pages
    ([1], [5000], 64, 2, 1, 64, 0),                           # one sequence for all warps
    ([1], [3000], 64, 8, 1, 128, 2500),
    # several scans of 32 sequences, with sequences without tokens and without keys
    ([(7 * i) % 3 for i in range(75)], [(7 * i) % 3 * (1 + 13 * i % 50) for i in range(75)], 16,
     4, 2, 64, 19),
    ([1] * 100, [1 + 37 * i % 90 for i in range(100)], 16, 2, 2, 128, 0),
    ([0] * 40 + [1], [0] * 40 + [33], 16, 2, 1, 64, 0),
    # clusters of eight, four and two blocks to a (sequence, head), and a block to each; page
    # borders, prefix borders and row fragments inside a warp's groups
    ([1, 1], [700, 1], 16, 16, 8, 64, 333),
    ([3, 2, 1], [300, 40, 7], 16, 16, 2, 128, 1001),
    ([1] * 5, [17, 400, 33, 90, 1], 16, 64, 8, 128, 17),
    ([1] * 40, [1 + 29 * i % 200 for i in range(40)], 16, 8, 4, 64, 40),
    ([2] * 37, [2 + 31 * i % 150 for i in range(37)], 16, 8, 8, 64, 0),
    ([2, 0, 1], [50, 0, 90], 3, 4, 2, 128, 100),
    ([1] * 2500, [1 + 5 * i % 23 for i in range(2500)], 16, 1, 1, 64, 5),  # many sequences
    # 17 to 32 rows over many keys: the tile kernel at D = 128, for own keys, the prefix, or both
    ([8, 8], [1500, 8], 64, 8, 2, 128, 0),
    ([5, 6, 5], [1030, 40, 5], 16, 8, 2, 128, 11),
    ([1, 1, 1], [40, 3, 200], 16, 16, 2, 128, 33000),
    ([20], [1025], 16, 2, 2, 128, 0),
    ([8, 1, 1, 1], [1200, 30, 0, 1100], 16, 8, 2, 128, 70),
    ([6, 6], [1100, 1030], 5, 8, 2, 128, 17),
    # long and short runs of new tokens in one batch: some behind few, some behind many rows
    ([1, 1, 1, 100], [50, 300, 1, 100], 16, 8, 2, 128, 0),
    ([200, 1, 0, 4, 5, 1], [230, 77, 0, 4, 300, 2000], 64, 8, 2, 64, 0),
    ([1, 70, 16, 17, 1, 1], [20, 70, 16, 90, 1, 0], 16, 1, 1, 128, 40),
    ([1] * 9 + [300] + [3] * 9, [40 + 50 * i for i in range(9)] + [301] + [5] * 9, 32, 14, 2, 64, 200),
    ([2, 1, 150, 0, 1], [9, 700, 1100, 0, 33], 128, 32, 1, 128, 0),       # 32 heads per kv head
    ([1, 129, 1, 1], [200, 129, 3, 40], 8, 24, 1, 64, 19),
    ([1] * 40 + [66] + [1] * 40, [1 + 7 * i for i in range(40)] + [66] + [3] * 40, 16, 4, 4, 64, 0),
    ([0] * 33 + [90] + [1] * 1200, [0] * 33 + [90] + [1 + i % 9 for i in range(1200)], 16, 2, 1, 64, 3),
    # the same with more than 32 heads per kv head: all of them behind many rows
    ([1, 1, 0, 1, 40], [50, 300, 0, 1, 45], 16, 48, 1, 64, 0),
    ([1] * 40 + [30] + [2] * 3, [1 + 7 * i for i in range(40)] + [66] + [3] * 3, 64, 64, 1, 128, 40),
    ([0, 9, 1, 1], [5, 9, 1, 500], 8, 128, 1, 64, 0),
    ([1, 1, 1, 17], [1500, 3, 0, 700], 128, 80, 2, 128, 0),
]


@pytest.mark.parametrize("case", range(len(PREFIX)))
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_prefix_attention(ra_lib, case, out_dtype):
    n, lens, page, hq, hkv, d, plen = PREFIX[case]
    x = Batch(n, lens, page, hkv, d, plen, seed=10 * case)
    q = randn(x.N, hq, d, seed=10 * case + 7)
    o, l = ra_lib.prefix_attn_fwd(q.to(DEV), *x.gpu("kp", "vp", "cu", "lens", "tables"), max(n),
                                  max_len=max(max(lens), 1), prefix_table=x.ptable.to(DEV),
                                  prefix_len=plen, out_dtype=out_dtype)
    assert ra_lib.ra_sync_status() == 0
    want = ref.prefix_attention(q, x.kp, x.vp, x.cu, x.lens, x.tables, x.ptable, plen, d ** -0.5)
    ref.check_attention(o, l.t(), (want[0], want[1], want[2].t()), f"case {case}")


RAGGED = [  # one or a few long runs of new tokens among short ones, where the rows kernel takes all
    ([1] * 20 + [150] + [1] * 7, [30 + i for i in range(20)] + [170] + [9] * 7, 24, 8, 2, 64, 0),
    ([0, 1, 90, 0, 2, 61, 0, 0, 1], [0, 700, 90, 0, 2, 100, 5, 0, 1], 5, 4, 4, 128, 31),
    ([1] * 300 + [77], [1 + i % 40 for i in range(300)] + [99], 48, 2, 1, 128, 50),
    ([2, 1, 1, 33, 1], [40, 3, 1000, 40, 1], 16, 130, 1, 64, 20),
    ([1, 1, 1, 9, 1, 1, 1, 1], [2000, 3, 1500, 9, 1, 0, 4000, 700], 64, 2, 2, 64, 0),  # one tile each
    ([0] * 30 + [1] * 8 + [4], [9, 0] * 15 + [60] * 8 + [700], 16, 8, 2, 64, 3000),  # prefix by tiles
    ([0] * 30 + [1] * 4 + [3], [9, 0] * 15 + [60] * 4 + [700], 48, 3, 1, 128, 500),  # and by rows
]


@pytest.mark.parametrize("case", range(len(RAGGED)))
@pytest.mark.parametrize("width", [1, 3000])
def test_ragged_batches_of_the_rows_kernel(ra_lib, case, width):
    """Row tiles and the combine's rows counted by token rows; rows of no sequence, before the
    first and behind the last, stay."""
    n, lens, page, hq, hkv, d, plen = RAGGED[case]
    x = Batch([3] + n, [3] + lens, page, hkv, d, plen, seed=7 * case, extra_rows=2)
    q = randn(x.N, hq, d, seed=case)
    q[:3] = q[-2:] = NAN
    wide = torch.cat([x.tables, torch.full((len(lens) + 1, width), 1 << 29, dtype=torch.int32)], 1)
    o = torch.full((x.N, hq, d), 7.0, device=DEV)
    l = torch.full((hq, x.N), 7.0, device=DEV)
    kp, vp, cu, lens_, pt = x.gpu("kp", "vp", "cu", "lens", "ptable")
    ra_lib.prefix_attn_fwd(q.to(DEV), kp, vp, cu[1:].clone(), lens_[1:].clone(),
                           wide[1:].contiguous().to(DEV), max(n), prefix_table=pt, prefix_len=plen,
                           out=o, lse=l)
    assert ra_lib.ra_sync_status() == 0
    for rows in (slice(0, 3), slice(x.N - 2, None)):
        assert (o[rows] == 7).all() and (l[:, rows] == 7).all()
    want = ref.prefix_attention(q[:-2], x.kp, x.vp, x.cu[1:], x.lens[1:], x.tables[1:], x.ptable,
                                plen, d ** -0.5)
    ref.check_attention(o[3:-2], l[:, 3:-2].t(), (want[0][3:], want[1][3:], want[2].t()[3:]),
                        f"case {case}")


def test_prompt_among_single_tokens_over_odd_pages(ra_lib):
    """255 single tokens and a prompt of 2000 whose tables could hold half a million keys: by
    B times the longest run that is a line of 4e9 groups of keys and was refused."""
    n, lens = [1] * 255 + [2000], [1 + 7 * i % 90 for i in range(255)] + [2000]
    x = Batch(n, lens, 24, 2, 128, seed=3, fill=0.0)
    wide = torch.zeros(256, 21846, dtype=torch.int32)
    wide[:, :x.max_pages] = x.tables.clamp(max=x.n_pages - 1)
    q = randn(x.N, 8, 128, seed=1)
    kp, vp, cu, lens_ = x.gpu("kp", "vp", "cu", "lens")
    o, l = ra_lib.prefix_attn_fwd(q.to(DEV), kp, vp, cu, lens_, wide.to(DEV), 2000)
    assert ra_lib.ra_sync_status() == 0
    want = ref.prefix_attention(q, x.kp, x.vp, x.cu, x.lens, x.tables, x.ptable, 0, 128 ** -0.5)
    ref.check_attention(o, l.t(), (want[0], want[1], want[2].t()), "prompt")


def test_ragged_token_rows_out_of_bounds_are_reported(ra_lib):
    """As below, where the combine finds the sequences and nobody else looks at them all."""
    x = Batch([1, 1, 40, 1, 1, 1], [9, 30, 60, 1, 5, 9], 24, 1, 64, seed=6, fill=0.0)
    q = randn(x.N, 1, 64, seed=2).to(DEV)
    kp, vp, lens_, tables = x.gpu("kp", "vp", "lens", "tables")

    def run(cu):
        ra_lib.prefix_attn_fwd(q, kp, vp, i32(cu).to(DEV), lens_, tables, 40)
        return ra_lib.load().ra_sync_status(None)

    good = x.cu.tolist()
    assert run(good) == 0
    for at, bad in ((-1, x.N + 1), (-1, 1 << 30), (-1, -(1 << 31)), (0, -5), (0, -(1 << 31)),
                    (1, x.N + 7), (1, (1 << 31) - 1), (1, -1)):
        cu = list(good)
        cu[at] = bad
        assert run(cu) == 5, cu
    assert run([0, x.N, 0, x.N, 0, x.N, 0]) == 5 and run(good) == 0


@pytest.mark.parametrize("n,lens", [([1, 1], [20, 3]), ([1] * 40, [9] * 40), ([70, 2], [75, 9])])
def test_bounds_far_above_the_lengths(ra_lib, n, lens):
    """Without max_len the tables' capacity is the bound: far above the lengths here, which
    are what is read."""
    x = Batch(n, lens, 64, 2, 64, 70, seed=9)
    wide = torch.cat([x.tables, torch.full((len(n), 4000), 1 << 29, dtype=torch.int32)], 1)
    q = randn(x.N, 4, 64, seed=1)
    kp, vp, cu, lens_, pt = x.gpu("kp", "vp", "cu", "lens", "ptable")
    o, l = ra_lib.prefix_attn_fwd(q.to(DEV), kp, vp, cu, lens_, wide.to(DEV), max(n) + 100,
                                  prefix_table=pt, prefix_len=70)
    assert ra_lib.ra_sync_status() == 0
    want = ref.prefix_attention(q, x.kp, x.vp, x.cu, x.lens, x.tables, x.ptable, 70, 0.125)
    ref.check_attention(o, l.t(), (want[0], want[1], want[2].t()), "wide")


def test_rows_that_see_nothing(ra_lib):
    """New tokens whose sequence has no key (length 0) and no prefix: 0 and -inf; a length
    below the token count leaves the first tokens without own keys."""
    x = Batch([2, 3, 1], [0, 2, 5], 16, 2, 64)
    q = randn(x.N, 4, 64, seed=3)
    o, l = ra_lib.prefix_attn_fwd(q.to(DEV), *x.gpu("kp", "vp", "cu", "lens", "tables"), 3,
                                  max_len=5)
    want = ref.prefix_attention(q, x.kp, x.vp, x.cu, x.lens, x.tables, x.ptable, 0, 0.125)
    assert (want[2][:, :3] == -float("inf")).all()
    ref.check_attention(o, l.t(), (want[0], want[1], want[2].t()), "empty")


def test_padded_batch_rows_stay(ra_lib):
    """Rows behind the last sequence are left as they were, in every output."""
    for plen in (0, 40):
        x = Batch([1, 2], [20, 30], 16, 2, 64, plen, extra_rows=5)
        q = randn(x.N, 4, 64, seed=5)
        q[3:] = NAN
        o = torch.full((x.N, 4, 64), 7.0, device=DEV)
        l = torch.full((4, x.N), 7.0, device=DEV)
        ra_lib.prefix_attn_fwd(q.to(DEV), *x.gpu("kp", "vp", "cu", "lens", "tables"), 2,
                               max_len=30, prefix_table=x.ptable.to(DEV), prefix_len=plen, out=o,
                               lse=l)
        assert (o[3:] == 7).all() and (l[:, 3:] == 7).all()
        want = ref.prefix_attention(q[:3], x.kp, x.vp, x.cu, x.lens, x.tables, x.ptable, plen,
                                    0.125)
        ref.check_attention(o[:3], l[:, :3].t(), (want[0], want[1], want[2].t()), "padded")


def test_padded_batch_rows_stay_with_many_tokens(ra_lib):
    """The same where the tensor-core tiles take the rows: a tile that reaches into the next
    sequence's rows, or into padding full of NaN, keeps to its own."""
    x = Batch([33, 50], [40, 77], 16, 2, 64, 150, extra_rows=70, seed=3)
    q = randn(x.N, 4, 64, seed=5)
    q[83:] = NAN
    o = torch.full((x.N, 4, 64), 7.0, device=DEV).bfloat16()
    l = torch.full((4, x.N), 7.0, device=DEV)
    ra_lib.prefix_attn_fwd(q.to(DEV), *x.gpu("kp", "vp", "cu", "lens", "tables"), 50, max_len=77,
                           prefix_table=x.ptable.to(DEV), prefix_len=150, out=o, lse=l)
    assert (o[83:] == 7).all() and (l[:, 83:] == 7).all()
    want = ref.prefix_attention(q[:83], x.kp, x.vp, x.cu, x.lens, x.tables, x.ptable, 150, 0.125)
    ref.check_attention(o[:83], l[:, :83].t(), (want[0], want[1], want[2].t()), "padded tiles")


@pytest.mark.parametrize("n,plen", [([3, 1, 2, 1], 0), ([3, 1, 2, 1], 20000), ([40, 30, 50, 33], 0),
                                    ([40, 30, 50, 33], 150), ([20, 20, 1, 1], 20000),
                                    ([2, 9, 1, 90], 0), ([90, 2, 120, 1], 300)])
def test_slice_of_a_batch(ra_lib, n, plen):
    """The last two sequences of a batch, given with all of its token rows: the rows of the
    others stay as they were, in the append too, whichever kernel takes the rows."""
    x = Batch(n, [m + 9 * i + 300 for i, m in enumerate(n)], 16, 2, 64, plen, extra_rows=3, seed=8)
    at, end = int(x.cu[2]), int(x.cu[4])
    q = randn(x.N, 4, 64, seed=5)
    q[:at] = q[end:] = NAN
    o = torch.full((x.N, 4, 64), 7.0, device=DEV)
    l = torch.full((4, x.N), 7.0, device=DEV)
    kp, vp, cu, lens, tables, pt = x.gpu("kp", "vp", "cu", "lens", "tables", "ptable")
    meta = (cu[2:].clone(), lens[2:].clone(), tables[2:].clone())
    ra_lib.prefix_attn_fwd(q.to(DEV), kp, vp, *meta, max(n[2:]), prefix_table=pt, prefix_len=plen,
                           out=o, lse=l)
    assert ra_lib.ra_sync_status() == 0
    for rows in (slice(0, at), slice(end, None)):
        assert (o[rows] == 7).all() and (l[:, rows] == 7).all()
    want = ref.prefix_attention(q[:end], x.kp, x.vp, x.cu[2:], x.lens[2:], x.tables[2:], x.ptable,
                                plen, 0.125)
    ref.check_attention(o[at:end], l[:, at:end].t(),
                        (want[0][at:], want[1][at:], want[2].t()[at:]), "slice")
    kv = randn(x.N, 2, 64, seed=6).to(DEV)
    whole = vp.clone()
    q_out = torch.full_like(q, 7.0).to(DEV)
    ra_lib.paged_kv_append(q.to(DEV), kv, kv, kp, vp, *meta, None, max(n[2:]), q_out=q_out)
    assert (q_out[:at] == 7).all() and (q_out[end:] == 7).all()
    assert torch.equal(q_out[at:end], q[at:end].to(DEV))
    for b in (0, 1):  # the other sequences' pages are not touched
        used = tables[b, :-(-int(x.lens[b]) // 16)].long()
        assert torch.equal(vp[used].nan_to_num(9e9), whole[used].nan_to_num(9e9))


@pytest.mark.parametrize("Lq", [1, 200])
def test_cross_key_counts_out_of_bounds(ra_lib, Lq):
    """A key count past the states is cut to them and reported; a negative one is none."""
    q, k, v = randn(2, Lq, 2, 64, seed=1), randn(2, 70, 2, 64, seed=2), randn(2, 70, 2, 64, seed=3)
    o, l = ra_lib.cross_attn_fwd(q.to(DEV), k.to(DEV), v.to(DEV), i32([71, -3]).to(DEV))
    assert ra_lib.load().ra_sync_status(None) == 5 and ra_lib.load().ra_sync_status(None) == 0
    want = ref.cross_attention(q, k, v, [70, 0], 0.125)
    ref.check_attention(o, l.transpose(1, 2), (want[0], want[1], want[2].transpose(1, 2)), "cut")


def test_two_calls_at_once(ra_lib):
    """Calls on two streams at the same time, and the host's next call before the last has
    run, do not meet in each other's workspace."""
    x = Batch([1] * 20 + [40], [50 + 9 * i for i in range(20)] + [90], 16, 2, 64, 300, seed=2)
    args = [(randn(x.N, 4, 64, seed=i).to(DEV), *x.gpu("kp", "vp", "cu", "lens", "tables"), 40)
            for i in range(2)]
    kw = dict(max_len=221, prefix_table=x.ptable.to(DEV), prefix_len=300)
    want = [ra_lib.prefix_attn_fwd(*a, **kw) for a in args]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in args]
    got = []
    for _ in range(10):
        got += [(i, ra_lib.prefix_attn_fwd(*args[i], stream=streams[i], **kw)) for i in range(2)]
    torch.cuda.synchronize()
    for i, (o, l) in got:
        assert torch.equal(o, want[i][0]) and torch.equal(l, want[i][1])


def test_strided_queries_and_interleaved_pages(ra_lib):
    """q as a slice of a wider projection; K and V pages interleaved in one allocation."""
    x = Batch([3, 1], [50, 20], 16, 2, 64, 40, seed=2)
    wide = randn(x.N, 10, 64, seed=9)
    q = wide[:, 1:5]
    kv = torch.stack([x.kp, x.vp], 1).to(DEV)
    o, l = ra_lib.prefix_attn_fwd(wide.to(DEV)[:, 1:5], kv[:, 0], kv[:, 1],
                                  *x.gpu("cu", "lens", "tables"), 3, max_len=50,
                                  prefix_table=x.ptable.to(DEV), prefix_len=40)
    want = ref.prefix_attention(q, x.kp, x.vp, x.cu, x.lens, x.tables, x.ptable, 40, 0.125)
    ref.check_attention(o, l.t(), (want[0], want[1], want[2].t()), "strided")


def test_large_scores_and_extremes(ra_lib):
    """Scores of some hundreds (one key takes nearly all the weight), and the same bits on
    every call."""
    x = Batch([2, 1], [70, 300], 16, 2, 64, 100, seed=4, fill=0.0)
    q = randn(x.N, 4, 64, seed=1) * 64
    args = (q.to(DEV), *x.gpu("kp", "vp", "cu", "lens", "tables"), 2)
    kw = dict(max_len=300, prefix_table=x.ptable.to(DEV), prefix_len=100)
    o, l = ra_lib.prefix_attn_fwd(*args, **kw)
    o2, l2 = ra_lib.prefix_attn_fwd(*args, **kw)
    assert torch.equal(o, o2) and torch.equal(l, l2)
    # the scores' error grows with them: 64 times the unit case's 5.5e-5 is 3.5e-3, in the
    # exponent, so a relative error of the weights of 2 * 3.5e-3 on top of the bf16 step
    want = ref.prefix_attention(q, x.kp, x.vp, x.cu, x.lens, x.tables, x.ptable, 100, 0.125)
    tol = (ref.U + 7e-3) * (want[1] + want[0].abs())
    assert ((o.double().cpu() - want[0]).abs() <= tol).all()
    assert ((l.double().cpu() - want[2]).abs() <= 3.5e-3 + 2.0 ** -20 * want[2].abs()).all()


def test_visible_nan_comes_through(ra_lib):
    """A NaN in a key that a row sees is not swallowed by the softmax."""
    x = Batch([1, 1], [40, 40], 16, 1, 64, seed=6)
    x.kp[int(x.tables[0, 1]), 3] = NAN
    q = randn(2, 1, 64, seed=2)
    o, l = ra_lib.prefix_attn_fwd(q.to(DEV), *x.gpu("kp", "vp", "cu", "lens", "tables"), 1,
                                  max_len=40)
    assert torch.isnan(o[0]).all() and torch.isnan(l[:, 0]).all()
    assert torch.isfinite(o[1]).all() and torch.isfinite(l[:, 1]).all()


def test_indices_out_of_bounds_are_reported(ra_lib):
    """Page ids, lengths and token counts outside their bounds are not followed; the next
    ra_sync_status says so, once."""
    x = Batch([1, 1], [20, 30], 16, 1, 64, seed=6, fill=0.0)
    q = randn(2, 1, 64, seed=2).to(DEV)
    k, v = randn(2, 1, 64, seed=3).to(DEV), randn(2, 1, 64, seed=4).to(DEV)
    kp, vp, cu, lens, tables = x.gpu("kp", "vp", "cu", "lens", "tables")

    def run(**kw):
        a = dict(cu=cu, lens=lens, tables=tables) | kw
        ra_lib.prefix_attn_fwd(q, kp, vp, a["cu"], a["lens"], a["tables"], 1, max_len=30)
        first = ra_lib.load().ra_sync_status(None)
        ra_lib.paged_kv_append(q, k, v, kp.clone(), vp.clone(), a["cu"], a["lens"], a["tables"],
                               None, 1)
        second = ra_lib.load().ra_sync_status(None)
        assert ra_lib.load().ra_sync_status(None) == 0
        return first, second

    assert run() == (0, 0)
    bad = tables.clone()
    bad[1, 1] = x.n_pages
    assert run(tables=bad) == (5, 5)
    bad[1, 1] = -1
    assert run(tables=bad) == (5, 5)
    assert run(lens=i32([20, 33]).to(DEV)) == (5, 5)
    assert run(lens=i32([20, 1 << 30]).to(DEV)) == (5, 5)
    assert run(cu=i32([0, 2, 2]).to(DEV)) == (5, 5)
    # a row count that is not sorted is cut at the tensor's rows
    run(cu=i32([0, 1, 1 << 30]).to(DEV))
    run(cu=i32([-5, 1, 2]).to(DEV))


@pytest.mark.parametrize("n,lens", [([1, 1], [20, 30]), ([1, 1], [20, 20000]),
                                    ([300, 1, 1], [320, 20, 20]), ([300, 300], [320, 320])])
def test_a_bad_index_beside_a_wait_that_ran_out(ra_lib, n, lens):
    """Both are reported, the wait first (the ring kernel's test hook withholds a load)."""
    x = Batch(n, lens, 16, 1, 64, seed=6, fill=0.0)
    q = randn(x.N, 1, 64, seed=2).to(DEV)
    kp, vp, cu, lens_, tables = x.gpu("kp", "vp", "cu", "lens", "tables")
    ring = [torch.zeros(s, dtype=torch.bfloat16, device=DEV) for s in
            [(1, 256, 1, 64), (1, 1, 256, 1, 64), (1, 1, 256, 1, 64)]]
    old = ra_lib.ra_set_wait_limit_ns(20_000_000)
    try:
        ra_lib.ra_debug_inject_stall(True)
        ra_lib.ring_attn_fwd(*ring, False)
        bad = tables.clone()
        bad[0, 0] = x.n_pages
        ra_lib.prefix_attn_fwd(q, kp, vp, cu, lens_, bad, max(n), max_len=max(lens))
        status = [ra_lib.load().ra_sync_status(None) for _ in range(3)]
    finally:
        ra_lib.ra_set_wait_limit_ns(old)
    assert status == [4, 5, 0]


@pytest.mark.parametrize("lens,width", [([20, 30], 1), ([20, 30], 4000), ([80, 50], 1),
                                        ([80, 50, 9, 9], 1)])
def test_token_rows_out_of_bounds_are_reported(ra_lib, lens, width):
    """Token rows past the tensors' or below 0, and counts above their bound or below 0, in
    each kernel: clusters, rows (the bound on the lengths far above them), tiles, both."""
    m = 40 if lens[0] == 80 else 1
    n = ([m, m] if len(lens) == 2 else [m, 1, 1, 1])
    N = sum(n)
    x = Batch(n, lens, 16, 1, 64, seed=6, fill=0.0)
    q, k, v = (randn(N, 1, 64, seed=i).to(DEV) for i in (2, 3, 4))
    kp, vp, lens_, tables = x.gpu("kp", "vp", "lens", "tables")
    wide = torch.cat([tables] + [tables[:, :1]] * width, 1)

    def run(cu):
        cu = i32(cu).to(DEV)
        ra_lib.prefix_attn_fwd(q, kp, vp, cu, lens_, wide, m)
        first = ra_lib.load().ra_sync_status(None)
        ra_lib.paged_kv_append(q, k, v, kp.clone(), vp.clone(), cu, lens_, tables, None, m)
        return first, ra_lib.load().ra_sync_status(None)

    good = x.cu.tolist()
    assert run(good) == (0, 0)
    for at, bad in ((-1, N + 1), (-1, 1 << 30), (-1, -(1 << 31)), (0, -5), (0, -(1 << 31)),
                    (1, N + 7), (1, (1 << 31) - 1), (1, -1)):
        cu = list(good)
        cu[at] = bad
        assert run(cu) == (5, 5), cu
    if m == 1:
        assert run([0, 2, 2]) == (5, 5)


APPEND = [  # n, lens, page, hq, hkv, d, rot, interleaved, offset
    ([1], [1], 16, 4, 2, 64, 64, False, 0),
    ([1, 1, 1], [1, 17, 200], 16, 8, 2, 128, 128, False, 32768),
    ([5, 0, 12, 1], [5, 0, 30, 9], 16, 4, 4, 64, 32, True, 1000003),
    ([33, 2], [40, 2], 64, 6, 2, 128, 64, True, 7),
    ([9], [9], 5, 2, 1, 64, 48, False, 123),
    ([3, 4], [8, 4], 1, 7, 1, 128, 16, False, 2000000000),
    ([6], [6], 16, 4, 2, 64, 0, False, 0),
    ([130], [131], 32, 0, 3, 128, 128, False, 5),
    # few sequences with many tokens: blocks over the rows, whatever their sequences
    ([1] * 40 + [99] + [2] * 40, [3 + 5 * i for i in range(40)] + [99] + [2] * 40, 16, 4, 2, 64, 64,
     False, 77),
    ([0, 1, 301, 0, 0, 1, 3, 2], [0, 400, 311, 0, 5, 1, 3, 9], 64, 24, 8, 128, 64, True, 0),
    ([1] * 1100 + [50], [1 + i % 3 for i in range(1100)] + [60], 5, 0, 1, 64, 32, False, 9),
    ([50, 1, 1, 1], [50, 9, 9, 1], 16, 1, 1, 64, 16, False, 0),                      # one warp
]


@pytest.mark.parametrize("case", range(len(APPEND)))
def test_append(ra_lib, case):
    n, lens, page, hq, hkv, d, rot, inter, offset = APPEND[case]
    x = Batch(n, lens, page, hkv, d, seed=20 * case, extra_rows=2)
    wide = randn(x.N, hq + 2 * hkv, d, seed=3)
    inv = (10000.0 ** (-torch.arange(0, rot, 2) / max(rot, 1))).float() if rot else None
    dev = wide.to(DEV)
    q, k, v = dev[:, :hq], dev[:, hq:hq + hkv], dev[:, hq + hkv:]
    kp, vp = x.kp.to(DEV), x.vp.to(DEV)
    q_out = torch.full((x.N, hq, d), 7.0, device=DEV).bfloat16() if hq else None
    got = ra_lib.paged_kv_append(q if hq else None, k, v, kp, vp,
                                 *x.gpu("cu", "lens", "tables"),
                                 inv.to(DEV) if rot else None, max(n), pos_offset=offset,
                                 interleaved=inter, q_out=q_out)
    assert ra_lib.ra_sync_status() == 0
    own = torch.cat([torch.arange(ln - m, ln) for m, ln in zip(n, lens)])
    pos = own + offset
    T = len(own)
    rk = ref.rotate(wide[:T, hq:hq + hkv], pos, inv, inter)
    want_k, want_v = x.kp.double(), x.vp.double()
    size_k = torch.zeros_like(want_k)
    half = rot // 2
    i = torch.arange(half)
    a, b = (2 * i, 2 * i + 1) if inter else (i, i + half)

    def pair_size(t):  # |x| + |y| of the rotated pairs
        z = torch.zeros(t.shape, dtype=torch.float64)
        t = t.double().abs()
        z[..., a] = z[..., b] = t[..., a] + t[..., b]
        return z

    sk = pair_size(wide[:T, hq:hq + hkv])
    t = 0
    for s, m in enumerate(n):
        for _ in range(m):
            w = (int(x.tables[s, int(own[t]) // page]), int(own[t]) % page)
            want_k[w], want_v[w], size_k[w] = rk[t], wide[t, hq + hkv:].double(), sk[t]
            t += 1
    # every row of the cache: the written ones within half a bf16 step (plus the fp32 sine's
    # and products' error, 2^-20 of the pair), all others and V bit for bit
    assert torch.equal(vp.double().cpu().nan_to_num(9e9), want_v.nan_to_num(9e9))

    def close(got, want, size):
        got, want = got.double().cpu(), want
        assert torch.equal(got.isnan(), want.isnan())
        err = (got - want).abs().nan_to_num(0)
        tol = (ref.U * (1 + 2.0 ** -10) * want.abs().nan_to_num(0) + 2.0 ** -20 * size)
        tol[size == 0] = 0  # copied elements
        assert (err <= tol).all(), float((err - tol).max())

    close(kp, want_k, size_k)
    if hq:
        close(got[:T], ref.rotate(wide[:T, :hq], pos, inv, inter), pair_size(wide[:T, :hq]))
        assert (got[T:] == 7).all()
    else:
        assert got is None


def test_append_of_a_very_long_run(ra_lib):
    """One run of 2^20 tokens among 4095 single ones: more than 2^31 places by sequence."""
    page, B, run = 256, 4096, 1 << 20
    lens = torch.ones(B, dtype=torch.int32)
    lens[7] = run
    cu = torch.cat([i32([0]), lens.cumsum(0).int()])
    N, pages = int(cu[-1]), B - 1 + run // page
    ids = torch.randperm(pages, generator=torch.Generator().manual_seed(1)).int()
    tables = torch.full((B, run // page), 1 << 29, dtype=torch.int32)
    tables[7] = ids[B - 1:]
    tables[torch.arange(B) != 7, 0] = ids[:B - 1]
    k, v = randn(N, 1, 64, seed=1).to(DEV), randn(N, 1, 64, seed=2).to(DEV)
    kp, vp = torch.zeros(2, pages, page, 1, 64, dtype=torch.bfloat16, device=DEV)
    ra_lib.paged_kv_append(None, k, v, kp, vp, cu.to(DEV), lens.to(DEV), tables.to(DEV), None, run)
    assert ra_lib.ra_sync_status() == 0
    ids = ids.long().to(DEV)
    single = torch.cat([torch.arange(7), torch.arange(7 + run, N)]).to(DEV)
    for pool, x in ((kp, k), (vp, v)):
        assert torch.equal(pool[ids[B - 1:]].view(run, 1, 64), x[7:7 + run])
        assert torch.equal(pool[ids[:B - 1], 0], x[single])
        assert not pool[ids[:B - 1], 1:].any()


def test_step_without_tokens(ra_lib):
    """A batch whose sequences bring no token: nothing is written, the results are empty."""
    x = Batch([0, 0], [5, 40], 16, 2, 64, 20)
    kp, vp, cu, lens, tables, pt = x.gpu("kp", "vp", "cu", "lens", "tables", "ptable")
    before = kp.clone(), vp.clone()
    q, k = (torch.empty(0, h, 64, dtype=torch.bfloat16, device=DEV) for h in (4, 2))
    r = ra_lib.paged_kv_append(q, k, k, kp, vp, cu, lens, tables, torch.ones(32, device=DEV), 1)
    assert r.shape == (0, 4, 64) and r.dtype == torch.bfloat16
    assert ra_lib.paged_kv_append(None, k, k, kp, vp, cu, lens, tables, None, 1) is None
    o, l = ra_lib.prefix_attn_fwd(r, kp, vp, cu, lens, tables, 1, prefix_table=pt, prefix_len=20)
    assert o.shape == (0, 4, 64) and l.shape == (4, 0) and o.dtype == torch.float32
    assert all(torch.equal(a.nan_to_num(9e9), b.nan_to_num(9e9))
               for a, b in zip(before, (kp, vp)))
    with pytest.raises(ValueError):  # the checks are those of any call
        ra_lib.prefix_attn_fwd(r, kp, vp, cu.long(), lens, tables, 1)
    assert ra_lib.ra_sync_status() == 0


def test_append_in_place_query(ra_lib):
    x = Batch([3, 2], [9, 2], 16, 2, 64, seed=8)
    q, k, v = (randn(5, h, 64, seed=h).to(DEV) for h in (4, 2, 2))
    inv = torch.rand(32).to(DEV)
    kp, vp = x.kp.to(DEV), x.vp.to(DEV)
    args = (k, v, kp, vp, *x.gpu("cu", "lens", "tables"), inv, 3)
    want = ra_lib.paged_kv_append(q, *args)
    got = ra_lib.paged_kv_append(q, *args, q_out=q)
    assert got is q and torch.equal(q, want)


CROSS = [  # B, Lq, Lk, lens, hq, hkv, d
    (1, 1, 1, [1], 1, 1, 64),
    (3, 1, 50, [50, 0, 17], 4, 4, 64),
    (2, 1, 1500, [1500, 3], 8, 2, 128),
    (2, 3, 65, None, 6, 2, 64),
    (2, 17, 200, [200, 130], 4, 1, 128),
    (1, 130, 77, [70], 8, 8, 64),
    (2, 300, 129, [129, 128], 2, 2, 128),
    (3, 257, 640, [1, 0, 513], 7, 1, 64),
    (1, 40, 1100, [1029], 1, 1, 128),
    (2, 500, 64, [64, 63], 8, 2, 64),
    (1, 129, 2000, None, 2, 1, 64),
    (70, 1, 90, [(11 * b) % 91 for b in range(70)], 4, 2, 64),
    (40, 2, 200, [(50 * b) % 201 for b in range(40)], 2, 1, 128),
    (1, 1, 6000, [5999], 4, 1, 64),
]


def cross_inputs(case, seed=0):
    B, Lq, Lk, lens, hq, hkv, d = CROSS[case]
    q = randn(B, Lq, hq, d, seed=seed + 1)
    kv = randn(B, Lk, 2, hkv, d, seed=seed + 2)
    for b, n in enumerate(lens or []):
        kv[b, n:] = NAN
    return q, kv, lens


@pytest.mark.parametrize("case", range(len(CROSS)))
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_cross_attention(ra_lib, case, out_dtype):
    q, kv, lens = cross_inputs(case, 30 * case)
    dev = kv.to(DEV)
    o, l = ra_lib.cross_attn_fwd(q.to(DEV), dev[:, :, 0], dev[:, :, 1],
                                 kv_lens=i32(lens).to(DEV) if lens else None,
                                 out_dtype=out_dtype)
    assert ra_lib.ra_sync_status() == 0
    want = ref.cross_attention(q, kv[:, :, 0], kv[:, :, 1], lens or [kv.shape[1]] * q.shape[0],
                               q.shape[-1] ** -0.5)
    ref.check_attention(o, l.transpose(1, 2), (want[0], want[1], want[2].transpose(1, 2)),
                        f"case {case}")


def test_decoder_step_together(ra_lib):
    """Three decoder steps as a model runs them: append, attention behind the prefix over
    the cache that the append filled, cross attention to the encoder's states."""
    hq, hkv, d, page, plen = 4, 2, 64, 16, 37
    x = Batch([0, 0, 0], [0, 0, 0], page, hkv, d, plen, seed=5, spare_pages=9, fill=0.0)
    free = [p for p in range(x.n_pages) if p not in x.ptable.tolist()]
    tables = i32(free[:6]).view(3, 2)
    lens = i32([0, 0, 0])
    kp, vp, pt = x.gpu("kp", "vp", "ptable")
    inv = (10000.0 ** (-torch.arange(0, d, 2) / d)).float()
    enc = randn(3, 29, 2, hkv, d, seed=50)
    enc_len = [29, 1, 14]
    ck, cv = x.kp.clone(), x.vp.clone()
    for step, n in enumerate(([5, 1, 14], [1, 1, 1], [1, 1, 1])):
        lens = lens + i32(n)
        cu = i32([0, n[0], n[0] + n[1], sum(n)])
        qkv = randn(sum(n), hq + 2 * hkv, d, seed=60 + step)
        dev = qkv.to(DEV)
        meta = (cu.to(DEV), lens.to(DEV), tables.to(DEV))
        q = ra_lib.paged_kv_append(dev[:, :hq], dev[:, hq:hq + hkv], dev[:, hq + hkv:], kp, vp,
                                   *meta, inv.to(DEV), max(n), pos_offset=plen)
        o, l = ra_lib.prefix_attn_fwd(q, kp, vp, *meta, max(n), prefix_table=pt, prefix_len=plen,
                                      out_dtype=torch.bfloat16)
        want = ref.prefix_attention(q.cpu(), kp.cpu(), vp.cpu(), cu, lens, tables, x.ptable, plen,
                                    d ** -0.5)
        ref.check_attention(o, l.t(), (want[0], want[1], want[2].t()), f"step {step}")
        if step:
            e = enc.to(DEV)
            c, cl = ra_lib.cross_attn_fwd(o[:, None], e[:, :, 0], e[:, :, 1],
                                          kv_lens=i32(enc_len).to(DEV))
            w = ref.cross_attention(o.cpu()[:, None], enc[:, :, 0], enc[:, :, 1], enc_len,
                                    d ** -0.5)
            ref.check_attention(c, cl.transpose(1, 2), (w[0], w[1], w[2].transpose(1, 2)), "cross")
    # the cache holds every token's rotated key: the attention above read what was appended
    own = kp.cpu()[tables[2].long()].flatten(0, 1)[:16]
    assert (own != 0).any(-1).all() and torch.equal(kp.cpu()[x.ptable.long()],
                                                    ck[x.ptable.long()])


def test_side_stream_and_graph(ra_lib):
    """On another stream than the current one, and captured: the graph follows device
    lengths and tables that change between replays, and two graphs run side by side."""
    x = Batch([1, 1], [20, 33], 16, 2, 64, 20, seed=11, fill=0.0)
    q = randn(2, 4, 64, seed=12)
    kp, vp, cu, lens, tables, pt = x.gpu("kp", "vp", "cu", "lens", "tables", "ptable")
    qd = q.to(DEV)
    kw = dict(max_len=64, prefix_table=pt, prefix_len=20)
    wide = torch.cat([tables, tables], 1).contiguous()
    want, wl = ra_lib.prefix_attn_fwd(qd, kp, vp, cu, lens, wide, 1, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o, l = ra_lib.prefix_attn_fwd(qd, kp, vp, cu, lens, wide, 1, stream=side, **kw)
    side.synchronize()
    assert torch.equal(o, want) and torch.equal(l, wl)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            res = ra_lib.prefix_attn_fwd(qd, kp, vp, cu, lens, wide, 1, **kw)
        graphs.append((g, res))
    lens.copy_(i32([19, 7]))
    s2 = torch.cuda.Stream()
    torch.cuda.synchronize()
    graphs[0][0].replay()
    with torch.cuda.stream(s2):
        graphs[1][0].replay()
    torch.cuda.synchronize()
    x.lens = i32([19, 7])
    w = ref.prefix_attention(q, x.kp, x.vp, x.cu, x.lens, x.tables, x.ptable, 20, 0.125)
    for _, (o, l) in graphs:
        ref.check_attention(o, l.t(), (w[0], w[1], w[2].t()), "graph")


def test_offsets_past_32_bits(ra_lib):
    """Pages whose element offset is past 2^32: a page stride of 2^28 elements, 17 pages in
    one allocation of 9 GB, K and V interleaved; keys only in the last page."""
    page, hkv, d = 16, 2, 64
    stride = 1 << 28
    buf = torch.empty(16 * stride + 2 * page * hkv * d, dtype=torch.bfloat16, device=DEV)
    kv = buf.as_strided((17, 2, page, hkv, d), (stride, page * hkv * d, hkv * d, d, 1))
    k, v = randn(page, hkv, d, seed=1), randn(page, hkv, d, seed=2)
    qkv = randn(1, 4 + 2 * hkv, d, seed=3)
    kv[16, 0], kv[16, 1] = k.to(DEV), v.to(DEV)
    cu, lens, table = i32([0, 1]).to(DEV), i32([10]).to(DEV), i32([[16]]).to(DEV)
    dev = qkv.to(DEV)
    q = ra_lib.paged_kv_append(dev[:, :4], dev[:, 4:6], dev[:, 6:], kv[:, 0], kv[:, 1], cu, lens,
                               table, None, 1)
    o, l = ra_lib.prefix_attn_fwd(q, kv[:, 0], kv[:, 1], cu, lens, table, 1)
    assert ra_lib.ra_sync_status() == 0
    k[9], v[9] = qkv[0, 4:6], qkv[0, 6:]
    assert torch.equal(kv[16, 0].cpu(), k) and torch.equal(kv[16, 1].cpu(), v)
    w = ref.prefix_attention(qkv[:, :4], k[None], v[None], i32([0, 1]), i32([10]), i32([[0]]),
                             i32([]), 0, 0.125)
    ref.check_attention(o, l.t(), (w[0], w[1], w[2].t()), "far page")
