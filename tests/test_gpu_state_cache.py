"""Upkeep of the state cache on the GPU: copying, forking, counting and
compacting slots, against plain lists.  Everything is whole numbers and
copies, so every comparison is exact."""
import numpy as np
import pytest
import torch

from gated_deltanet_layer_causal_amd import capi as L
from gated_deltanet_layer_causal_amd.layer import CoreConfig, GDNStateCache
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu


def ints(v):
    return torch.tensor(np.asarray(v, dtype=np.int32), device=DEV)


def make(n_slots, words, seed):
    """A cache buffer [n_slots, words] int32 with distinct contents."""
    rng = np.random.default_rng(seed)
    data = rng.integers(-2**31, 2**31 - 1, (n_slots, words)).astype(np.int32)
    return data, torch.tensor(data, device=DEV)


def ws(n_slots):
    return torch.full((L.gdn_cache_workspace(n_slots),), 0xAB, dtype=torch.uint8, device=DEV)


def ref_fork(data, refs, src):
    data, refs = data.copy(), refs.copy()
    before = refs.copy()
    free = [i for i in range(len(refs)) if refs[i] == 0]
    dst = []
    for s in src:
        ok = s == -1 or (0 <= s < len(refs) and before[s] > 0)
        if not ok or not free:
            dst.append(-1)
            continue
        d = free.pop(0)
        dst.append(d)
        refs[d] = 1
        data[d] = data[s] if s >= 0 else 0
    return data, refs, dst


def ref_compact(data, refs, table):
    data, refs = data.copy(), refs.copy()
    live = [i for i in range(len(refs)) if refs[i] > 0]
    remap = [-1] * len(refs)
    holes = [i for i in range(len(live)) if refs[i] == 0]
    for i in live:
        if i < len(live):
            remap[i] = i
        else:
            h = holes.pop(0)
            remap[i] = h
            data[h], refs[h], refs[i] = data[i], refs[i], 0
    return data, refs, remap, [remap[t] if 0 <= t < len(refs) else t for t in table]


@pytest.mark.parametrize("n_slots,words,n,live", [
    (1, 4, 1, 0.0), (1, 4, 3, 1.0), (5, 8, 3, 0.5), (64, 4, 70, 0.3), (64, 4100, 9, 0.5),
    (1023, 4, 1025, 0.4), (1025, 4, 300, 0.9), (5000, 4, 2500, 0.5), (5000, 4, 7000, 0.1),
    (300, 4, 40, 1.0), (300, 20, 400, 0.0)])
def test_fork(n_slots, words, n, live):
    rng = np.random.default_rng(n_slots + n)
    data, buf = make(n_slots, words, 1)
    refs = (rng.random(n_slots) < live).astype(np.int32) * rng.integers(1, 4, n_slots).astype(np.int32)
    src = rng.integers(-3, n_slots + 2, n)
    src[rng.random(n) < 0.2] = -1
    if refs.any():
        alive = np.flatnonzero(refs)
        pick = rng.random(n) < 0.5
        src[pick] = rng.choice(alive, pick.sum())      # the same slot several times
    want, want_refs, want_dst = ref_fork(data, refs, src.tolist())
    t_refs, dst = ints(refs), ints(np.full(n, 77))
    L.gdn_cache_fork(buf, t_refs, ints(src), dst, ws(n_slots))
    assert dst.tolist() == want_dst
    assert t_refs.tolist() == want_refs.tolist()
    assert np.array_equal(buf.cpu().numpy(), want)


@pytest.mark.parametrize("n_slots,words,live", [
    (1, 4, 0.0), (1, 4, 1.0), (2, 8, 0.5), (7, 4, 0.5), (64, 4100, 0.4), (1024, 4, 0.5), (1025, 4, 0.2),
    (5000, 4, 0.6), (300, 4, 1.0), (300, 4, 0.0), (5000, 4, 0.02), (5000, 4, 0.98)])
def test_compact(n_slots, words, live):
    rng = np.random.default_rng(n_slots + words)
    data, buf = make(n_slots, words, 2)
    refs = (rng.random(n_slots) < live).astype(np.int32) * rng.integers(1, 4, n_slots).astype(np.int32)
    table = np.concatenate([rng.permutation(n_slots), rng.integers(-5, n_slots + 5, 1500)])
    want, want_refs, want_remap, want_table = ref_compact(data, refs, table.tolist())
    t_refs, remap, t_table = ints(refs), ints(np.full(n_slots, 55)), ints(table)
    L.gdn_cache_compact(buf, t_refs, remap, t_table, ws(n_slots))
    assert remap.tolist() == want_remap
    assert t_refs.tolist() == want_refs.tolist()
    assert t_table.tolist() == want_table
    assert np.array_equal(buf.cpu().numpy(), want)
    L.gdn_cache_compact(buf, t_refs, remap, None, ws(n_slots))      # again: nothing to move
    assert np.array_equal(buf.cpu().numpy(), want) and t_refs.tolist() == want_refs.tolist()


def test_counts():
    """Slots named several times in one call count several times; counts
    stop at 0; free slots and entries outside the cache are left alone."""
    refs = ints([0, 1, 2, 3, 1])
    L.gdn_cache_retain(refs, ints([0, 1, 1, 3, -1, 5, 1 << 30]))
    assert refs.tolist() == [0, 3, 2, 4, 1]
    L.gdn_cache_release(refs, ints([0, 1, 2, 2, 2, 3, 4, -7, 5]))
    assert refs.tolist() == [0, 2, 0, 3, 0]
    L.gdn_cache_release(refs, ints([1] * 1000 + [3]))
    assert refs.tolist() == [0, 0, 0, 2, 0]
    many = ints([1])
    L.gdn_cache_retain(many, ints([0] * 100000))
    assert many.tolist() == [100001]
    L.gdn_cache_retain(many, ints([]))
    assert many.tolist() == [100001]
    full = ints([2**31 - 2])
    L.gdn_cache_retain(full, ints([0] * 70))
    assert full.tolist() == [2**31 - 1]


@pytest.mark.parametrize("words", [4, 12, 1020, 4096, 4100, 50000])
def test_copy(words):
    a_h, a = make(6, words, 3)
    b_h, b = make(9, words, 4)
    src, dst = [5, -1, 2, 2, 6, 0, 3, 1 << 30], [0, 8, 4, 6, 2, -1, 9, 1]
    L.gdn_cache_copy(a, b, ints(src), ints(dst))
    want = b_h.copy()
    for s, d in zip(src, dst):
        if 0 <= d < 9:
            want[d] = 0 if s < 0 else -1 if s >= 6 else a_h[s]
    assert np.array_equal(b.cpu().numpy(), want)
    L.gdn_cache_copy(b, a, src_idx=ints([8, 7, 6, 5, 4, 3]))        # gather
    assert np.array_equal(a.cpu().numpy(), want[[8, 7, 6, 5, 4, 3]])
    c_h, c = make(3, words, 5)
    L.gdn_cache_copy(c, b, dst_idx=ints([4, -1, 0]))                # scatter
    want[4], want[0] = c_h[0], c_h[2]
    assert np.array_equal(b.cpu().numpy(), want)
    L.gdn_cache_copy(b, b, ints([4, 0]), ints([5, 6]))              # within one cache
    want[5], want[6] = want[4], want[0]
    assert np.array_equal(b.cpu().numpy(), want)


def test_copy_between_strides_leaves_the_gaps():
    """Layer views of two caches: only the slots' own bytes are touched."""
    cfg = CoreConfig(1, 2, 32, torch.bfloat16)
    a, b = GDNStateCache(cfg, 4, 2, DEV), GDNStateCache(cfg, 3, 1, DEV)
    a.buffer.random_(0, 255)
    b.buffer.random_(0, 255)
    before = b.buffer.clone()
    L.gdn_cache_copy(a.S(1), b.S(0), ints([3, 0]), ints([0, 2]))
    assert torch.equal(b.S(0)[[0, 2]].view(torch.int32), a.S(1)[[3, 0]].view(torch.int32))
    n = b.S(0)[0].numel() * 4
    assert torch.equal(b.buffer[1], before[1]) and torch.equal(b.buffer[:, n:], before[:, n:])
    L.gdn_cache_copy(a.conv(1), b.conv(0), ints([1]), ints([1]))
    assert torch.equal(b.conv(0)[1].view(torch.int16), a.conv(1)[1].view(torch.int16))


def test_a_day_of_a_cache():
    """Random forks, retains, releases and compactions in a row, the plain
    lists beside them."""
    rng = np.random.default_rng(9)
    cfg = CoreConfig(1, 2, 32, torch.bfloat16)
    cache = GDNStateCache(cfg, 37, 2, DEV)
    cache.buffer.random_(0, 255)
    data, refs = cache.buffer.view(torch.int32).cpu().numpy().copy(), np.zeros(37, np.int32)
    for k in range(40):
        what = rng.integers(0, 4)
        if what == 0:
            src = rng.integers(-2, 38, rng.integers(1, 12))
            data, refs, want = ref_fork(data, refs, src.tolist())
            assert cache.fork(ints(src)).tolist() == want, k
        elif what == 1:
            slots = rng.integers(-1, 38, 6)
            for s in slots:
                if 0 <= s < 37 and refs[s] > 0:
                    refs[s] += 1
            cache.retain(ints(slots))
        elif what == 2:
            slots = rng.integers(-1, 38, 15)
            for s in slots:
                if 0 <= s < 37:
                    refs[s] = max(refs[s] - 1, 0)
            cache.release(ints(slots))
        else:
            table = rng.integers(-1, 37, 20)
            data, refs, remap, want = ref_compact(data, refs, table.tolist())
            t = ints(table)
            assert cache.compact(t).tolist() == remap and t.tolist() == want, k
        assert cache.refs.tolist() == refs.tolist(), k
        assert np.array_equal(cache.buffer.view(torch.int32).cpu().numpy(), data), k


def test_captured_and_replayed():
    """A graph of release, compact and fork, replayed; each replay does what
    the eager calls do."""
    cfg = CoreConfig(1, 2, 32, torch.bfloat16)
    cache, twin = GDNStateCache(cfg, 12, 1, DEV), GDNStateCache(cfg, 12, 1, DEV)
    cache.buffer.random_(0, 255)
    cache.refs.copy_(ints([1] * 9 + [0] * 3))
    twin.buffer.copy_(cache.buffer)
    twin.refs.copy_(cache.refs)
    gone, src, table = ints([2, 5, 11]), ints([-1, 0, 7]), ints(list(range(9)))
    t2 = table.clone()

    def run(c, t):
        c.release(gone)
        remap = c.compact(t)
        return remap, c.fork(src)

    run(GDNStateCache(cfg, 12, 1, DEV), table.clone())     # loads the kernels
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(cache, table)
    for k in range(4):
        gone.copy_(ints([[2, 5, 11], [0, 1, 2], [8, 8, 3], [-1, 4, 10]][k]))
        graph.replay()
        torch.cuda.synchronize()
        want = run(twin, t2)
        assert got[0].tolist() == want[0].tolist() and got[1].tolist() == want[1].tolist(), k
        assert table.tolist() == t2.tolist() and cache.refs.tolist() == twin.refs.tolist(), k
        assert torch.equal(cache.buffer, twin.buffer), k


def test_slots_beyond_32_bit_offsets():
    gap = 3 << 30
    big = torch.empty(2 * gap + 4096, dtype=torch.uint8, device=DEV)
    far = torch.as_strided(big.view(torch.int32), (3, 1024), (gap // 4, 1))
    h, t = make(3, 1024, 6)
    L.gdn_cache_copy(t, far)
    L.gdn_cache_copy(far, far, ints([0]), ints([2]))
    back = torch.empty_like(t)
    L.gdn_cache_copy(far, back)
    assert np.array_equal(back.cpu().numpy(), h[[0, 1, 0]])
    wide = big[:2 * gap].view(torch.int32).view(2, -1)     # two slots of 3 GiB
    wide[0, ::1 << 20] = 7
    wide[0, -5:] = ints([1, 2, 3, 4, 5])
    refs, dst = ints([1, 0]), ints([9])
    L.gdn_cache_fork(wide, refs, ints([0]), dst, ws(2))
    assert dst.tolist() == [1] and torch.equal(wide[0], wide[1])
