"""Host side of the cache operators: every bad argument is refused before anything is
launched (the pointers below are never dereferenced), and the workspace sizes are sane."""
import ctypes

import pytest
import torch

FAKE = 0x10000
I64 = ctypes.c_longlong


@pytest.fixture(scope="module")
def lib():
    from sequence_parallelism_attn_b200 import build, ra
    build.build()
    return ra.load()


APPEND = dict(q=FAKE, k=FAKE, v=FAKE, qs=256, ks=128, vs=128, cu=FAKE, lens=FAKE, tables=FAKE,
              inv=FAKE, B=2, N=4, T=2, hq=4, hkv=2, d=64, rot=64, inter=0, off=0, page=16, n=8,
              mp=4, ps=2048, dt=0, qo=FAKE + 4096, qos=256, kp=FAKE, vp=FAKE)
PREFIX = dict(q=FAKE, qs=256, kp=FAKE, vp=FAKE, cu=FAKE, lens=FAKE, tables=FAKE, pt=FAKE, plen=20,
              B=2, N=4, T=2, max_len=64, hq=4, hkv=2, d=64, page=16, n=8, mp=4, ps=2048,
              scale=0.125, dt=0, odt=0, out=FAKE, lse=FAKE, ws=FAKE, wsb=1 << 40)
CROSS = dict(q=FAKE, k=FAKE, v=FAKE, lens=FAKE, B=2, Lq=3, Lk=50, hq=4, hkv=2, d=64, qt=256,
             qb=768, kt=128, kb=6400, scale=0.125, dt=0, odt=0, out=FAKE, lse=FAKE, ws=FAKE,
             wsb=1 << 40)


def call(lib, entry, base, kw):
    assert set(kw) <= set(base)
    args = list((base | kw).values())
    return getattr(lib, entry)(*args, None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=0), 1), (dict(k=FAKE + 8), 1), (dict(v=0), 1), (dict(qo=0), 1), (dict(kp=FAKE + 2), 1),
    (dict(cu=0), 1), (dict(lens=FAKE + 1), 1), (dict(tables=0), 1), (dict(inv=0), 1),
    (dict(qs=248), 1), (dict(qs=260), 1), (dict(ks=127), 1), (dict(vs=64), 1), (dict(qos=200), 1),
    (dict(B=0), 1), (dict(N=0), 1), (dict(T=0), 1), (dict(T=5), 1), (dict(hq=-1), 1),
    (dict(hq=3), 1), (dict(hkv=0), 1), (dict(rot=8), 1), (dict(rot=80), 1), (dict(rot=-16), 1),
    (dict(inter=2), 1), (dict(off=-1), 1), (dict(page=0), 1), (dict(n=0), 1), (dict(mp=0), 1),
    (dict(ps=2040), 1), (dict(ps=2049), 1), (dict(d=96), 2), (dict(dt=1), 2), (dict(dt=7), 1),
    (dict(N=1 << 25), 1), (dict(qo=FAKE, qos=512), 1), (dict(B=(1 << 28) + 1), 1),
])
def test_append_refusals(lib, kw, status):
    assert call(lib, "ra_paged_kv_append", APPEND, kw) == status
    assert lib.ra_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(q=0), 1), (dict(qs=264 - 16), 1), (dict(qs=257), 1), (dict(kp=0), 1),
    (dict(vp=FAKE + 4), 1), (dict(cu=FAKE + 2), 1), (dict(lens=0), 1), (dict(tables=0), 1),
    (dict(pt=0), 1), (dict(plen=-1), 1), (dict(B=0), 1), (dict(N=0), 1), (dict(T=9), 1),
    (dict(max_len=0), 1), (dict(max_len=65), 1), (dict(hq=5), 1), (dict(d=32), 2),
    (dict(page=0), 1), (dict(ps=100), 1), (dict(scale=0.0), 1), (dict(scale=float("inf")), 1),
    (dict(scale=float("nan")), 1), (dict(dt=1), 2), (dict(odt=3), 1), (dict(out=0), 1),
    (dict(lse=FAKE + 4), 1), (dict(ws=0, plen=1 << 17), 1), (dict(ws=FAKE + 8, plen=1 << 17), 1),
    (dict(wsb=16, plen=1 << 17), 1),
])
def test_prefix_refusals(lib, kw, status):
    assert call(lib, "ra_prefix_attn_fwd", PREFIX, kw) == status
    assert lib.ra_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(q=0), 1), (dict(k=FAKE + 8), 1), (dict(v=0), 1), (dict(lens=FAKE + 2), 1),
    (dict(B=0), 1), (dict(Lq=0), 1), (dict(Lk=0), 1), (dict(hq=3), 1), (dict(d=256), 2),
    (dict(qt=255), 1), (dict(qb=700), 1), (dict(kt=130), 1), (dict(kb=6392), 1),
    (dict(scale=-1.0), 1), (dict(dt=1), 2), (dict(odt=2), 1), (dict(out=FAKE + 2), 1),
    (dict(lse=0), 1), (dict(B=1 << 13, Lq=1 << 13, qb=1 << 21), 1),
])
def test_cross_refusals(lib, kw, status):
    assert call(lib, "ra_cross_attn_fwd", CROSS, kw) == status
    assert lib.ra_last_error()


def test_workspace_sizes(lib):
    lib.ra_prefix_attn_workspace.restype = I64
    # few rows over a moderate number of keys: one kernel, no partial results
    assert lib.ra_prefix_attn_workspace(4, 4, 1, 100, 0, 8, 2, 64, 16) == 0
    some = lib.ra_prefix_attn_workspace(4, 4, 1, 1 << 17, 0, 8, 2, 64, 16)
    assert 0 < some < lib.ra_prefix_attn_workspace(4, 4, 1, 1 << 17, 1000, 8, 2, 64, 16)
    assert lib.ra_prefix_attn_workspace(0, 4, 1, 100, 0, 8, 2, 64, 16) == 0
    # bounded by the resident warps, not by the keys
    assert lib.ra_prefix_attn_workspace(1, 1, 1, 1 << 24, 1 << 24, 32, 8, 128, 16) < 32 << 20
    # many rows in one range of keys: results are written without partials
    assert lib.ra_cross_attn_workspace(64, 300, 100, 8, 8, 64) == 0
    assert lib.ra_cross_attn_workspace(1, 30, 1000, 8, 2, 64) > 0
    assert lib.ra_cross_attn_workspace(1, 1, 1000, 8, 2, 64) == 0


def test_workspace_follows_the_tokens(lib):
    """A ragged batch of one long run of new tokens among many single ones: the workspace is in
    proportion to the rows, whatever the page size, not to B times the longest run."""
    def size(*a):
        return lib.ra_prefix_attn_workspace(*a)

    for B, new, hq, hkv, d in ((256, 2000, 32, 8, 128), (256, 8000, 32, 8, 128),
                               (65, 4000, 32, 8, 128), (256, 2000, 8, 8, 64)):
        n = B - 1 + new
        # a row's partial result, of whole tiles of 32 rows: those that n tokens fill, one more
        # to a sequence, one to each of the 1184 resident warps
        tiles = n * (hq // hkv) // 32 + B + 1184 // hkv + 1
        most = tiles * hkv * (32 * (d + 1) * 4 + 8) + 32
        for page in (1, 5, 24, 48, 96):
            assert 0 < size(B, n, new, new, 0, hq, hkv, d, page) <= most, (B, new, page)
            assert size(B, n, new, 1 << 17, 0, hq, hkv, d, page) <= most, (B, new, page)
    # sequences without tokens cost nothing
    assert size(1 << 16, 10, 1, 4000, 0, 32, 8, 128, 16) <= size(1 << 4, 10, 1, 4000, 0, 32, 8, 128, 16)


@pytest.mark.parametrize("kw", [
    # single tokens and one prompt, tables for 131072 keys, pages that the tile kernel does not take
    dict(B=256, N=2255, T=2000, hq=32, hkv=8, d=128, qs=4096, page=24, ps=24576, mp=5462,
         max_len=131072),
    # and one of a million tokens with 128 heads to a kv head
    dict(B=4096, N=(1 << 20) + 4095, T=1 << 20, hq=128, hkv=1, qs=8192, ps=1024, mp=1 << 16),
])
def test_ragged_batches_are_not_too_large(lib, kw):
    """What a launch would need follows the tokens: such a batch is refused for the workspace
    that is missing here, not for its size."""
    assert call(lib, "ra_prefix_attn_fwd", PREFIX, kw | dict(wsb=16)) == 1
    assert b"workspace" in lib.ra_last_error()


def test_native_module_is_rebuilt_for_another_torch(monkeypatch, tmp_path):
    from sequence_parallelism_attn_b200 import build
    runs = []

    def compile_(cmd, verbose):
        runs.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()

    monkeypatch.setattr(build, "_run", compile_)
    monkeypatch.setattr(build, "NATIVE", str(tmp_path / "_ra_torch.so"))
    monkeypatch.setattr(build, "BUILD_DIR", str(tmp_path / "_build"))
    for want in (1, 1):
        build.build_native()
        assert len(runs) == want
    monkeypatch.setattr(torch, "__version__", "0.0.0")
    for want in (2, 2):
        build.build_native()
        assert len(runs) == want
    build.build_native(force=True)
    assert len(runs) == 3


def test_native_module_is_loaded_once(monkeypatch):
    """Threads that ask for the native module at the same time get the same one, complete."""
    import threading
    import time

    from sequence_parallelism_attn_b200 import build, ra
    build.build()
    made = []

    class Loader:
        def __init__(self, name, path):
            pass

        def create_module(self, spec):
            made.append(type("Module", (), {})())
            return made[-1]

        def exec_module(self, module):
            time.sleep(0.05)
            module.set_error_class = lambda cls: setattr(module, "cls", cls)

    monkeypatch.setattr(ra, "_native", None)
    monkeypatch.setattr(ra.importlib.machinery, "ExtensionFileLoader", Loader)
    got, start = [], threading.Barrier(8)

    def ask():
        start.wait()
        m = ra.native()
        got.append((m, getattr(m, "cls", None)))

    threads = [threading.Thread(target=ask) for _ in range(8)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert len(made) == 1 and got == [(made[0], ra.RaError)] * 8


def test_binding_refusals():
    """The binding checks shapes, types and layouts before the library is called."""
    from sequence_parallelism_attn_b200 import ra
    nat = ra.native()
    bf = dict(dtype=torch.bfloat16)
    pages = torch.zeros(4, 16, 2, 64, **bf)
    inter = torch.zeros(4, 2, 16, 2, 64, **bf)
    assert nat.check_cache(inter[:, 0], inter[:, 1]) == (4, 16, 2, 64, 4096)
    assert nat.check_cache(pages[:1], pages[:1]) == (1, 16, 2, 64, 2048)
    for bad in ((pages, pages[:, :8]), (pages.float(), pages.float()), (pages, inter[:, 0]),
                (pages[..., ::2], pages[..., ::2]), (pages[:, :, :1], pages[:, :, :1]),
                (pages[0], pages[0])):
        with pytest.raises(ValueError):
            nat.check_cache(*bad)
    i32 = dict(dtype=torch.int32)
    cu, lens, tables = torch.zeros(4, **i32), torch.zeros(3, **i32), torch.zeros(3, 5, **i32)
    assert nat.check_batch(cu, lens, tables) == (3, 5)
    for bad in ((cu.long(), lens, tables), (cu[:3], lens, tables), (cu, lens[:2], tables),
                (cu, lens, tables[:, 0]), (cu, lens, tables[:, ::2]), (cu, lens.float(), tables)):
        with pytest.raises(ValueError):
            nat.check_batch(*bad)
    q, k = torch.zeros(2, 5, 4, 64, **bf), torch.zeros(2, 7, 2, 64, **bf)
    assert nat.check_cross(q, k, k, None) == (2, 5, 7, 4, 2, 64, 256, 1280, 128, 896)
    kv = torch.zeros(2, 7, 2, 2, 64, **bf)
    assert nat.check_cross(q, kv[:, :, 0], kv[:, :, 1], torch.zeros(2, **i32))[8:] == (256, 1792)
    for bad in ((q, k[:1], k[:1]), (q, k[..., :32], k[..., :32]), (q, k, k[:, :6]),
                (q.float(), k, k), (q.transpose(1, 2), k, k),
                (q, k, torch.zeros(2, 7, 4, 64, **bf)[:, :, :2])):
        with pytest.raises(ValueError):
            nat.check_cross(*bad, None)
    with pytest.raises(ValueError):
        nat.check_cross(q, k, k, torch.zeros(3, **i32))
    with pytest.raises(ValueError):
        ra.cross_attn_fwd(q, k, k)  # not on a GPU
    with pytest.raises(ValueError):
        ra.paged_kv_append(q[0], k[0], k[0], pages, pages, cu, lens, tables, None, 1)


CROSS_BWD = dict(q=FAKE, k=FAKE, v=FAKE, lens=FAKE, o=FAKE, lse=FAKE, do=FAKE, B=2, Lq=3, Lk=50,
                 hq=4, hkv=2, d=64, qt=256, qb=768, kt=128, kb=6400, scale=0.125, dt=0, gdt=0,
                 dq=FAKE, dk=FAKE, dv=FAKE, ws=FAKE, wsb=1 << 40)


@pytest.mark.parametrize("kw,status", [
    (dict(q=0), 1), (dict(k=0), 1), (dict(v=FAKE + 8), 1), (dict(lens=FAKE + 2), 1),
    (dict(o=0), 1), (dict(lse=0), 1), (dict(do=FAKE + 2), 1), (dict(dq=0), 1),
    (dict(dk=FAKE + 4), 1), (dict(dv=0), 1), (dict(ws=0), 1), (dict(wsb=100), 1),
    (dict(B=0), 1), (dict(Lq=0), 1), (dict(Lk=0), 1), (dict(hkv=3), 1), (dict(d=32), 2),
    (dict(qt=8), 1), (dict(qb=8), 1), (dict(kt=8), 1), (dict(kb=8), 1), (dict(scale=0.0), 1),
    (dict(dt=1), 2), (dict(gdt=2), 1),
])
def test_cross_backward_refusals(lib, kw, status):
    assert call(lib, "ra_cross_attn_bwd", CROSS_BWD, kw) == status
    assert lib.ra_last_error()


def test_cross_backward_workspace(lib):
    # Delta rows, and dQ in fp32 where the gradients are rounded to bf16
    assert lib.ra_cross_attn_bwd_workspace(2, 3, 4, 64, 1) == 4 * 24
    assert lib.ra_cross_attn_bwd_workspace(2, 3, 4, 64, 0) == 4 * 24 * 65


def test_reference_gradients_against_differences():
    """The 64-bit formula that the GPU's gradients are held to is the derivative of the
    64-bit forward, masked batch rows and grouped heads included."""
    import _kv_ref as ref
    g = torch.Generator().manual_seed(0)
    q, k, v, do = (torch.randn(2, n, h, 8, generator=g, dtype=torch.float64)
                   for n, h in ((3, 4), (5, 2), (5, 2), (3, 4)))
    lens = [5, 3]
    grads, _ = ref.cross_backward(q, k, v, lens, do, 0.3)
    for i in range(3):
        for at in [(0, 0, 0, 0), (1, 2, 1, 5), (0, 1, 1, 3)]:
            def loss(h):
                y = [t.clone() for t in (q, k, v)]
                y[i][at] += h
                return (ref.cross_attention(*y, lens, 0.3)[0] * do).sum()
            d = (loss(1e-5) - loss(-1e-5)) / 2e-5
            assert abs(d - grads[i][at]) <= 1e-8 * (1 + abs(d))
