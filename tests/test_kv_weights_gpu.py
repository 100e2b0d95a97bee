"""The weights that the attention kernels apply to V add up to one: they are rounded to bf16
before they meet V, and the sum that divides the output is that of the rounded ones.  Shown
where a sum of the unrounded ones would be off the most: equal values, and a single key that
takes most of the weight without being its tile's maximum when the running maximum was set."""
import pytest
import torch

import _kv_ref as ref
from test_kv_gpu import DEV, Batch, i32, randn

pytestmark = pytest.mark.gpu

CASES = [  # n, lens, page, hq, hkv, d, prefix
    ([1, 1], [300, 700], 16, 8, 2, 64, 333),              # clusters
    ([1] * 5, [2000, 400, 33, 90, 1], 16, 64, 8, 128, 0),
    ([1] * 60, [1 + 40 * i % 900 for i in range(60)], 16, 16, 4, 64, 0),   # rows
    ([40, 7], [1090, 50], 5, 4, 1, 128, 31),
    ([300], [1300], 64, 8, 2, 64, 0),                     # tiles
    ([300], [1300], 64, 8, 2, 128, 0),
    ([20], [1025], 16, 2, 2, 128, 2100),                  # one row tile, shared by two warpgroups
    ([50], [50], 16, 4, 1, 64, 1500),
    ([1, 1, 1, 100], [50, 1300, 1, 600], 16, 8, 2, 128, 0),  # rows and tiles
    ([1, 1, 1, 100], [50, 1300, 1, 600], 16, 8, 2, 64, 1000),
]


def attend(ra, x, q, n, lens):
    return ra.prefix_attn_fwd(q.to(DEV), *x.gpu("kp", "vp", "cu", "lens", "tables"), max(n),
                              max_len=max(lens), prefix_table=x.ptable.to(DEV), prefix_len=x.plen)


@pytest.mark.parametrize("case", range(len(CASES)))
def test_equal_values_come_through(ra_lib, case):
    """With the same value in every key the output is that value, but for the order of fp32
    sums.  Every term has the value's sign, so a sum of n terms of which at most m are added
    one after another is off by m 2^-22 at most (an addition in the tensor core truncates
    the smaller operands, four times the 2^-24 of a rounding): m = n / 16 steps of a product
    with V, up to 32 + n / 128 of the weights' sum, some 10 in the joins.  For n <= 3400 that is
    below (213 + 59 + 10) 2^-22 < 2^-13.  A divisor of unrounded weights gives some 2^-9."""
    n, lens, page, hq, hkv, d, plen = CASES[case]
    x = Batch(n, lens, page, hkv, d, plen, seed=10 * case, fill=0.0)
    value = randn(hkv, d, seed=10 * case + 5)
    x.vp[:] = value
    q = randn(x.N, hq, d, seed=10 * case + 7)
    o, _ = attend(ra_lib, x, q, n, lens)
    assert ra_lib.ra_sync_status() == 0
    want = value.double().repeat_interleave(hq // hkv, 0).expand(x.N, hq, d)
    err = ((o.double().cpu() - want).abs() / want.abs().clamp(min=1e-30)).max()
    assert err <= 2.0 ** -13, float(err)


@pytest.mark.parametrize("Lq,Lk,hq,hkv,d", [(300, 1200, 4, 4, 64), (300, 1200, 8, 2, 128),
                                            (33, 1200, 8, 2, 64), (1, 1200, 8, 8, 64)])
def test_equal_values_come_through_cross(ra_lib, Lq, Lk, hq, hkv, d):
    q, k = randn(2, Lq, hq, d, seed=1), randn(2, Lk, hkv, d, seed=2)
    value = randn(2, 1, hkv, d, seed=3)
    v = value.expand(2, Lk, hkv, d).contiguous()
    o, _ = ra_lib.cross_attn_fwd(q.to(DEV), k.to(DEV), v.to(DEV), i32([Lk, Lk - 7]).to(DEV))
    assert ra_lib.ra_sync_status() == 0
    want = value.double().repeat_interleave(hq // hkv, 2).expand(2, Lq, hq, d)
    err = ((o.double().cpu() - want).abs() / want.abs().clamp(min=1e-30)).max()
    assert err <= 2.0 ** -13, float(err)


FEW_KEYS = [
    ([1, 1], [200, 250], 16, 8, 2, 64, 0),
    ([1] * 60, [130 + 40 * i % 100 for i in range(60)], 16, 16, 4, 128, 0),
    ([40], [250], 5, 4, 1, 128, 0),
    ([99], [255], 64, 8, 2, 64, 0),
    ([99], [255], 64, 8, 2, 128, 0),
    ([99, 1, 1, 1], [230, 200, 180, 1], 16, 8, 2, 128, 0),
    ([60, 50], [60, 50], 32, 8, 4, 64, 250),
]


@pytest.mark.parametrize("case", range(len(FEW_KEYS)))
def test_a_key_that_dominates(ra_lib, case):
    """One key of each sequence, and of the prefix, has a score about 5 above the others'
    largest: it takes most of the weight, and is rounded alone.  Weights w_j (1 + e_j), |e_j| <= u = 2^-8, divided by
    their own sum, give an output off by |sum_j p_j e_j (v_j - out)| / (1 - u) at most, which is
    u (1 + 2 u) sum_j p_j |v_j - out|; the scores' part (2^-12) is that of _kv_ref, once for the
    weights and once for their sum, for scores up to twice its unit size."""
    n, lens, page, hq, hkv, d, plen = FEW_KEYS[case]
    x = Batch(n, lens, page, hkv, d, plen, seed=10 * case, fill=0.0)
    base = randn(d, seed=case)
    q = (base + 0.25 * randn(x.N, hq, d, seed=10 * case + 7)).bfloat16()
    big = (base.float() * 7.2 * d ** 0.5 / (base.float() ** 2).sum()).bfloat16()
    for table, m in [(x.ptable, plen)] + [(x.tables[b], m) for b, m in enumerate(lens)]:
        j = 128  # behind the keys that the running maximum is first set by
        if m > j:
            x.kp[int(table[j // page]), j % page] = big
            x.vp[int(table[j // page]), j % page] = 4.0
    o, _ = attend(ra_lib, x, q, n, lens)
    assert ra_lib.ra_sync_status() == 0
    o = o.double().cpu()
    g, scale = hq // hkv, d ** -0.5
    pk, pv = ref.paged_keys(x.kp, x.ptable, plen), ref.paged_keys(x.vp, x.ptable, plen)
    for b, (m, ln) in enumerate(zip(n, lens)):
        ok, ov = ref.paged_keys(x.kp, x.tables[b], ln), ref.paged_keys(x.vp, x.tables[b], ln)
        for i in range(0, m, max(1, m // 5)):
            see, t = ln - m + i + 1, int(x.cu[b]) + i
            k, v = torch.cat([pk, ok[:see]]), torch.cat([pv, ov[:see]])
            for h in range(hq):
                p = torch.softmax(k[:, h // g] @ q[t, h].double() * scale, 0)
                w = p @ v[:, h // g]
                spread = p @ (v[:, h // g] - w).abs()
                tol = (ref.U * (1 + 2 * ref.U) + 2.0 ** -11) * spread + 2.0 ** -13 * (
                    p @ v[:, h // g].abs())
                err = (o[t, h] - w).abs()
                assert (err <= tol + 1e-30).all(), (b, i, h, float((err / tol).max()))
