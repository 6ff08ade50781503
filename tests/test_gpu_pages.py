"""GPU parity of the page copies: bytes equal to a plain copy's in every format."""
import numpy as np
import pytest
import torch

from oracle import bs8
from speculative_verify_attention_q3kv_gb300 import _lib, api

pytestmark = pytest.mark.gpu

UNIT = {"q3": 2 * 256 * 112, "fp8": 2 * 65536, "t5k": 256 * 276, "bs8": 2 * 65600}     # bytes per page, layer and kv head
CALL = {"q3": api.copy_pages, "fp8": api.fp8_copy_pages, "t5k": api.t5k_copy_pages, "bs8": api.bs8_copy_pages}


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def i32(v):
    return torch.tensor(np.asarray(v, np.int32)).cuda()


def _kept(fmt, rows):
    """Which bytes of a unit belong to its first `rows` positions."""
    at = np.arange(UNIT[fmt])
    if fmt in ("q3", "fp8"):
        return at % (UNIT[fmt] // 2) < rows * (UNIT[fmt] // 512)
    if fmt == "t5k":
        return np.where(at < 256 * 164, at < rows * 164, at - 256 * 164 < rows * 112)
    one = np.zeros(bs8.UNIT_BYTES, bool)
    one[bs8._OFFSETS[:rows].ravel()] = True
    one[bs8.CODE_BYTES:bs8.CODE_BYTES + 4 * ((rows + 15) // 16)] = True
    return np.concatenate([one, one])


def _pool(fmt, layers, kv, pages, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(0, 256, (pages * layers * kv * UNIT[fmt],), dtype=torch.uint8, generator=g, device="cuda")


def _copied(fmt, src_pool, dst_pool, units, src, dst, rows):
    """The destination pool as it should be."""
    a = src_pool.cpu().numpy().reshape(-1, units, UNIT[fmt])
    b = dst_pool.cpu().numpy().reshape(-1, units, UNIT[fmt]).copy()
    out = b.copy()
    for s, d, r in zip(src, dst, rows):
        out[d] = np.where(_kept(fmt, r)[None, :], a[s], b[d])
    return out.reshape(-1)


@pytest.mark.parametrize("fmt", list(UNIT))
@pytest.mark.parametrize("layers,kv", [(1, 1), (3, 2), (2, 5)])
def test_whole_and_partial_pages(fmt, layers, kv):
    rng = np.random.default_rng(layers)
    desc, pool = api.make_desc(layers, kv, 40), _pool(fmt, layers, kv, 40, kv)
    order = rng.permutation(40)
    src, dst = order[:15], order[15:30]
    rows = np.array([0, 1, 2, 7, 8, 9, 15, 16, 17, 31, 100, 128, 200, 255, 256])
    want = _copied(fmt, pool, pool, layers * kv, src, dst, rows)
    status = i32([0])
    CALL[fmt](desc, pool, i32(src), i32(dst), rows=i32(rows), status=status)
    assert np.array_equal(pool.cpu().numpy(), want) and int(status) == 0
    want = _copied(fmt, pool, pool, layers * kv, src, dst, [256] * 15)
    CALL[fmt](desc, pool, i32(src), i32(dst), status=status)
    assert np.array_equal(pool.cpu().numpy(), want) and int(status) == 0


@pytest.mark.parametrize("fmt", list(UNIT))
def test_into_another_pool(fmt):
    desc = api.make_desc(2, 2, 9)
    a, b = _pool(fmt, 2, 2, 9, 1), _pool(fmt, 2, 2, 5, 2)
    # page ids of the two pools have nothing to do with one another: one source may go to two places
    src, dst, rows = [8, 8, 0, 4], [0, 4, 1, 3], [256, 30, 255, 1]
    want, before = _copied(fmt, a, b, 4, src, dst, rows), a.clone()
    status = i32([0])
    CALL[fmt](desc, a, i32(src), i32(dst), rows=i32(rows), dst_pool=b, dst_num_pages=5, status=status)
    assert np.array_equal(b.cpu().numpy(), want) and torch.equal(a, before) and int(status) == 0
    CALL[fmt](desc, a, i32([1, 2]), i32([5, 2]), dst_pool=b, dst_num_pages=5, status=status)
    want = _copied(fmt, a, torch.from_numpy(want), 4, [2], [2], [256])
    assert np.array_equal(b.cpu().numpy(), want) and int(status) == _lib.Q3KV_STATUS_BAD_PAGE


def test_pairs_that_do_not_fit_together_are_skipped():
    desc, pool = api.make_desc(1, 1, 12), _pool("q3", 1, 1, 12, 3)

    def run(src, dst, rows=None):
        p, status = pool.clone(), i32([0])
        api.copy_pages(desc, p, i32(src), i32(dst), rows=None if rows is None else i32(rows), status=status)
        return p, int(status)

    def same(p, src, dst, rows=None):
        return np.array_equal(p.cpu().numpy(), _copied("q3", pool, pool, 1, src, dst, [256] * len(src) if rows is None else rows))

    p, s = run([0, 1, 2], [5, 5, 6])                  # one destination twice: neither is written
    assert s == 4 and same(p, [2], [6])
    p, s = run([0, 1, 2], [1, 7, 8])                  # a destination that another pair reads: that pair still reads the old page
    assert s == 4 and same(p, [1, 2], [7, 8])
    p, s = run([0, 1], [1, 0])                        # an exchange
    assert s == 4 and same(p, [], [])
    p, s = run([3, 4], [3, 9])                        # onto itself: nothing to do
    assert s == 0 and same(p, [4], [9])
    p, s = run([3, 4], [3, 3])                        # and over a page that is copied onto itself
    assert s == 4 and same(p, [], [])
    p, s = run([-1, 12, 0, 1, 2], [3, 4, -1, 12, 5])
    assert s == 4 and same(p, [2], [5])
    p, s = run([0, 1, 2], [3, 4, 5], [-1, 257, 100])
    assert s == 8 and same(p, [2], [5], [100])
    p, s = run([2, 2, 2], [3, 4, 5])                  # one source, several forks
    assert s == 0 and same(p, [2, 2, 2], [3, 4, 5])
    p, s = run([], [])
    assert s == 0 and torch.equal(p, pool)


def test_as_many_pairs_as_a_call_takes():
    desc, pool = api.make_desc(1, 1, 8192), _pool("q3", 1, 1, 8192, 4)
    g = torch.Generator().manual_seed(5)
    order = torch.randperm(8192, generator=g).numpy()
    src, dst = order[:4096], order[4096:]
    v = pool.view(8192, -1)
    want = v.clone()
    want[torch.from_numpy(dst).cuda()] = v[torch.from_numpy(src).cuda()]
    status = i32([0])
    api.copy_pages(desc, pool, i32(src), i32(dst), status=status)
    assert torch.equal(v, want) and int(status) == 0
    with pytest.raises(_lib.Q3KVError):
        api.copy_pages(desc, pool, i32(np.zeros(4097)), i32(np.zeros(4097)))


def test_pages_beyond_32_bit_offsets():
    desc = api.make_desc(16, 4, 640)                  # 8.4 MB a page
    pool = torch.empty(api.bs8_pool_bytes(desc), dtype=torch.uint8, device="cuda").view(640, -1)
    pool[600:].random_(0, 256)
    want = pool[631].clone()
    api.bs8_copy_pages(desc, pool.view(-1), i32([631]), i32([639]))
    assert torch.equal(pool[639], want) and torch.equal(pool[631], want)


def test_a_captured_copy_reads_its_lists_anew():
    desc, pool = api.make_desc(2, 2, 10), _pool("t5k", 2, 2, 10, 6)
    src, dst, rows = i32([0, 1]), i32([2, 3]), i32([256, 256])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        api.t5k_copy_pages(desc, pool, src, dst, rows=rows)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        api.t5k_copy_pages(desc, pool, src, dst, rows=rows)
    for a, b, r in (([4, 5], [6, 7], [200, 3]), ([6, 6], [8, 9], [13, 256])):
        want = _copied("t5k", pool, pool, 4, a, b, r)
        src.copy_(i32(a))
        dst.copy_(i32(b))
        rows.copy_(i32(r))
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(pool.cpu().numpy(), want)
