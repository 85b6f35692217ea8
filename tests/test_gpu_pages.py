"""The pages of the paged caches on the GPU: forks, room for new tokens with
copies on write, release, page copies and compaction, against plain forms."""
import random

import numpy as np
import pytest
import torch

import video_diffusion_kv_gb300 as qvg

from _pages import Pool

pytestmark = pytest.mark.gpu
BAD, FULL, OK = qvg.QVG_ERR_INVALID_ARG, qvg.QVG_ERR_CAPACITY, qvg.QVG_OK


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    yield
    assert qvg.get_status() == qvg.QVG_OK


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Both:
    """A pool, table and lengths on the GPU and their plain form, kept in step."""

    def __init__(self, pages, B, columns, page):
        self.plain = Pool(pages, B, columns, page)
        self.page, self.B = page, B
        self.pool = qvg.PagePool(pages)
        self.table = torch.zeros(B, columns, dtype=torch.int32, device="cuda")
        self.len = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.args = (self.pool, page, self.table, self.len)

    def same(self):
        assert self.pool.refs.tolist() == self.plain.refs and self.len.tolist() == self.plain.len
        for b, n in enumerate(self.plain.len):
            m = self.plain.pages(n)
            assert self.table[b, :m].tolist() == self.plain.table[b][:m], b

    def fork(self, parents, children):
        qvg.pages_fork(*self.args, ints(parents), ints(children))
        self.plain.fork(parents, children)

    def release(self, ids, keep=None):
        qvg.pages_release(*self.args, ints(ids), keep=None if keep is None else ints(keep))
        self.plain.release(ids, keep)

    def reserve(self, new):
        cu = ints([0] + list(np.cumsum(new)))
        slots, copies = qvg.pages_reserve(*self.args, cu_new=cu, total=sum(new))
        want = self.plain.reserve(new)
        if want is None:
            assert qvg.get_status() == FULL
            assert (slots == -1).all() and (copies == -1).all()
            return None
        assert slots.tolist() == want[0] and [tuple(x) for x in copies.tolist()] == want[1]
        return slots, copies


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("seed", range(4))
def test_random_runs(page, seed):
    """Random forks, growth, cuts and releases; at the end every page is free."""
    r = random.Random(100 * page + seed)
    B = r.choice((1, 3, 20, 70))
    b = Both(r.choice((5, 60, 200)), B, 9, page)
    for _ in range(25):
        op = r.choice(("grow", "grow", "fork", "release", "cut"))
        if op == "grow":
            b.reserve([r.choice((0, 0, 1, 3, page, 2 * page + 5)) if r.random() < 0.4 else 0 for _ in range(B)])
        elif op == "fork":
            empty = [i for i in range(B) if b.plain.len[i] == 0]
            r.shuffle(empty)
            some = empty[:r.randint(0, len(empty))]
            parents = [i for i in range(B) if i not in some]
            if some and parents:
                b.fork([r.choice(parents) for _ in some], some)
        else:
            ids = r.sample(range(B), r.randint(1, B))
            b.release(ids, None if op == "release" else [r.randint(0, b.plain.len[i]) for i in ids])
        b.same()
        assert qvg.get_status() == OK
    b.release(list(range(B)))
    b.same()
    assert not any(b.plain.refs)


@pytest.mark.parametrize("B,F,new", [(1, 1, 1), (2, 5, 1), (7, 3, 40), (300, 3, 2), (1500, 1, 1)])
def test_writers_of_a_shared_page(B, F, new):
    """Of a beam's writers each takes a copy while another holder is left: with
    the parent writing too, the last one keeps the page; without, all copy."""
    page = 16
    for parents_too in (True, False):
        b = Both(B * (F + 2) * (2 + new // page) + 3, B * (F + 1), 6, page)
        b.reserve([5 + i % 20 for i in range(B)] + [0] * (B * F))
        b.fork(list(range(B)) * F, list(range(B, B * (F + 1))))
        got = b.reserve([new if parents_too else 0] * B + [new] * (B * F))
        b.same()
        copied = int((got[1][:, 0] >= 0).sum())
        partly = sum((5 + i % 20) % page != 0 for i in range(B))
        assert copied == partly * F
    assert qvg.get_status() == OK


def test_large_pool_many_tokens():
    """Prompts of thousands of tokens (slots in a grid of their own), a pool
    whose free pages begin far behind, sequences that need nothing."""
    b = Both(70001, 40, 900, 64)
    b.reserve([50000] * 20 + [0] * 20)
    got = b.reserve([0] * 20 + [i * 13 for i in range(20)])
    b.same()
    assert len(got[0]) == 13 * 190
    b.release([3, 17, 5])
    b.reserve([1, 0, 7, 5000] + [0] * 35 + [30000])
    b.same()
    assert qvg.get_status() == OK


def test_uniform_growth_and_no_growth():
    b = Both(40, 5, 4, 16)
    slots, copies = qvg.pages_reserve(*b.args, n_new=17)
    want = b.plain.reserve([17] * 5)
    assert slots.tolist() == want[0] and (copies == -1).all()
    slots, copies = qvg.pages_reserve(*b.args, n_new=0)
    assert slots.numel() == 0 and (copies == -1).all()
    b.same()
    empty = torch.zeros(0, dtype=torch.int32, device="cuda")
    slots, copies = qvg.pages_reserve(b.pool, 16, b.table[:0], b.len[:0])
    assert slots.numel() == 0 and copies.shape == (0, 2)
    qvg.pages_fork(*b.args, empty, empty)
    qvg.pages_release(*b.args, empty)
    b.same()


def test_no_room():
    """Too few pages, and a row that is too short: nothing changes."""
    b = Both(6, 3, 4, 16)
    b.reserve([40, 16, 0])
    assert b.reserve([0, 16, 17]) is None  # 3 pages wanted, 2 free
    b.same()
    assert b.reserve([30, 0, 0]) is None  # 5 columns wanted, 4 there
    b.same()
    assert b.reserve([0, 5000, 0]) is None  # (slots in a grid of their own)
    b.same()
    assert b.reserve([8, 16, 16]) is not None
    b.same()
    assert qvg.get_status() == OK


def test_an_invalid_argument_comes_before_a_lack_of_room():
    """Whichever sequence has which, also where one thread meets both."""
    B = 1030
    for bad, long in ((0, 1024), (1024, 0), (3, 4)):
        pool, table, lens = qvg.PagePool(8), torch.zeros(B, 2, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
        lens[bad], lens[long] = -1, 32  # (a row of two pages of 16 is full)
        before = lens.clone()
        slots, copies = qvg.pages_reserve(pool, 16, table, lens)
        assert qvg.get_status() == BAD
        assert (slots == -1).all() and (copies == -1).all() and torch.equal(lens, before) and not pool.refs.any()
        lens[bad] = 0
        slots, copies = qvg.pages_reserve(pool, 16, table, lens)
        assert qvg.get_status() == qvg.QVG_ERR_CAPACITY and (slots == -1).all()


def test_more_than_a_billion_sequences():
    """Twice a sequence's number, and the sum of two, pass 31 bits: the last
    one's copy on write, and a batch without room."""
    B = 2 ** 30 + 5
    pool = qvg.PagePool(8)
    table, lens = torch.zeros(B, 1, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    cu = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    lens[[0, B - 1]], cu[B], pool.refs[0] = 5, 1, 2
    slots, copies = qvg.pages_reserve(pool, 16, table, lens, cu_new=cu, total=1)
    assert qvg.get_status() == OK
    assert slots.tolist() == [16 + 5] and copies[B - 1].tolist() == [0, 1] and (copies[:B - 1] == -1).all()
    assert lens[[0, B - 2, B - 1]].tolist() == [5, 0, 6] and table[B - 1].tolist() == [1] and pool.refs.tolist() == [1, 1] + [0] * 6
    del cu, slots, copies
    slots, copies = qvg.pages_reserve(pool, 16, table, lens)
    assert qvg.get_status() == FULL
    assert (slots == -1).all() and (copies == -1).all() and lens[B - 1].item() == 6


def test_bad_arguments_on_the_device():
    b = Both(30, 6, 4, 16)
    b.reserve([20, 5, 40, 0, 0, 0])
    before = (b.pool.refs.clone(), b.table.clone(), b.len.clone())

    def unchanged():
        return all(torch.equal(x, y) for x, y in zip(before, (b.pool.refs, b.table, b.len)))
    for parents, children in (([0], [1]), ([0], [6]), ([-1], [3]), ([0], [-2]), ([3], [3]), ([0, 1], [3, 3]), ([3, 0], [4, 3])):
        qvg.pages_fork(*b.args, ints(parents), ints(children))
        assert qvg.get_status() == BAD, (parents, children)
        if children == [4, 3]:  # an empty parent that is a child too: the child is refused, the other pair holds
            assert b.len.tolist() == [20, 5, 40, 0, 0, 0]
        assert unchanged()
    for ids, keep in (([6], None), ([-1], None), ([1, 1], None), ([0], [21]), ([0], [-1])):
        qvg.pages_release(*b.args, ints(ids), keep=None if keep is None else ints(keep))
        assert qvg.get_status() == BAD and unchanged(), ids
    for cu, total in (([0, 1, 2, 3, 4, 5, 7], 6), ([1, 1, 2, 3, 4, 5, 6], 6), ([0, 2, 1, 3, 4, 5, 6], 6), ([0, 1, 2, 3, 4, 5, 5], 6)):
        slots, copies = qvg.pages_reserve(*b.args, cu_new=ints(cu), total=total)
        assert qvg.get_status() == BAD and unchanged(), cu
        assert (slots == -1).all() and (copies == -1).all()
    b.table[1, 0] = 30  # a last page outside the pool
    slots, _ = qvg.pages_reserve(*b.args)
    assert qvg.get_status() == BAD and (slots == -1).all() and torch.equal(b.len, before[2])
    b.table.copy_(before[1])
    b.pool.refs[b.table[2, 1].item()] = 0  # held by nobody: passed over, the others given back
    qvg.pages_release(*b.args, ints([2]))
    assert qvg.get_status() == BAD and b.len.tolist() == [20, 5, 0, 0, 0, 0]
    assert int(b.pool.refs.sum()) == 3 and int(b.pool.refs.min()) == 0
    b.len[0] = -4
    qvg.pages_release(*b.args, ints([0]))
    assert qvg.get_status() == BAD and b.len[0].item() == -4


def test_in_a_graph_and_on_streams():
    """A captured step (cut to the accepted length, room for two tokens)
    replayed on a changing state; two pools at once on two streams."""
    b = Both(64, 4, 8, 16)
    b.reserve([20, 31, 16, 1])
    ids, keep = ints([0, 1, 2, 3]), ints([20, 31, 16, 1])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qvg.pages_release(*b.args, ids, keep=keep)
        slots, copies = qvg.pages_reserve(*b.args, n_new=2)
    for _ in range(5):
        now = [n - 1 if i % 2 else n for i, n in enumerate(b.plain.len)]
        keep.copy_(ints(now))
        graph.replay()
        b.plain.release([0, 1, 2, 3], now)
        want = b.plain.reserve([2] * 4)
        assert slots.tolist() == want[0] and (copies == -1).all()
        b.same()
    sides = [(torch.cuda.Stream(), Both(300, 30, 8, 16)) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(6):
        for s, x in sides:
            got = qvg.pages_reserve(*x.args, n_new=7, stream=s)
            x.last = got, x.plain.reserve([7] * 30)
    torch.cuda.synchronize()
    for _, x in sides:
        x.same()
        assert x.last[0][0].tolist() == x.last[1][0]


def caches(page, pages, seed):
    """One of each kind, filled with random bytes (latents: random numbers)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    got = []
    for H, d, bits in ((3, 128, 8), (1, 64, 8), (2, 128, 4), (5, 64, 4)):
        c = qvg.PagedKV(H, d, page, pages, bits)
        for t in (c.k_codes, c.k_scales, c.v_codes, c.v_scales):
            t.copy_(torch.randint(0, 256, t.shape, generator=g, device="cuda", dtype=torch.uint8))
        got.append((c, [c.k_codes, c.k_scales, c.v_codes, c.v_scales], 2))
    for dc, dr in ((256, 64), (64, 0), (192, 24), (128, 8)):
        c = qvg.LatentKV(dc, dr, page, pages)
        for t in (c.c, c.kr):
            t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
        got.append((c, [c.c, c.kr], 1))
    return got


@pytest.mark.parametrize("page", [16, 64, 256])
def test_copy(page):
    for c, buffers, _ in caches(page, 12, page):
        before = [t.clone() for t in buffers]
        pairs = [(0, 11), (-1, -1), (3, 5), (3, 6), (-1, 4), (7, -1), (1, 2)]
        qvg.pages_copy(c, ints(pairs))
        for t, was in zip(buffers, before):
            for a, b in pairs:
                if a >= 0 and b >= 0:
                    was[b] = was[a]
            assert torch.equal(t, was)
        assert qvg.get_status() == OK
        qvg.pages_copy(c, ints([(12, 0), (0, 12), (4, 9)]))
        assert qvg.get_status() == BAD
        for t, was in zip(buffers, before):
            was[9] = was[4]
            assert torch.equal(t, was)
        qvg.pages_copy(c, torch.zeros(0, 2, dtype=torch.int32, device="cuda"))


def test_copy_of_many_pairs():
    c = qvg.LatentKV(64, 0, 16, 140010)
    c.c.copy_(torch.arange(140010, device="cuda")[:, None, None] % 251)
    pairs = torch.stack((torch.arange(70000), torch.arange(70000) + 70005), 1).int().cuda()
    qvg.pages_copy(c, pairs)
    assert torch.equal(c.c[70005:140005], c.c[:70000]) and (c.c[140005:] == (torch.arange(140005, 140010, device="cuda") % 251)[:, None, None]).all()


def test_copy_of_more_than_a_billion_pairs():
    """Twice a pair's number passes 31 bits."""
    n = 2 ** 30 + 3
    c = qvg.LatentKV(64, 0, 16, 8)
    c.c.copy_(torch.arange(8, device="cuda")[:, None, None])
    pairs = torch.full((n, 2), -1, dtype=torch.int32, device="cuda")
    pairs[1], pairs[2 ** 30], pairs[n - 1] = ints([0, 4]), ints([1, 5]), ints([2, 6])
    qvg.pages_copy(c, pairs)
    assert qvg.get_status() == OK
    assert c.c[:, 0, 0].tolist() == [0, 1, 2, 3, 0, 1, 2, 7]


@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("lens,share", [((1, 40, 700), 0.5), ((2000, 3), 0.9), ((513, 512, 511, 0), 0.1), ((900,), 1.0)])
def test_compact(page, lens, share):
    """Every kept token's bytes at their new place, the first ones and what no
    kept token moves to as they were."""
    r = random.Random(page + len(lens))
    pages = sum(-(-n // page) for n in lens) + 2
    order = r.sample(range(pages), pages)
    table, at = np.zeros((len(lens), max(1, max(-(-n // page) for n in lens))), np.int32), 0
    for b, n in enumerate(lens):
        m = -(-n // page)
        table[b, :m] = order[at:at + m]
        at += m
    first = [r.randint(0, min(n, 20)) for n in lens]
    kept = [sorted(r.sample(range(f, n), int((n - f) * share))) for f, n in zip(first, lens)]
    keep = np.full((len(lens), max(1, max(map(len, kept)))), -5, np.int32)
    for b, k in enumerate(kept):
        keep[b, :len(k)] = k
    for c, buffers, off in caches(page, pages, 7):
        before = [t.clone() for t in buffers]
        qvg.paged_compact(c, ints(table), ints(first), ints(keep), ints([len(k) for k in kept]))
        assert qvg.get_status() == OK
        for t, was in zip(buffers, before):
            want = was.clone()
            rows, old = (x.transpose(1, 2) if off == 2 else x for x in (want, was))
            for b, k in enumerate(kept):
                if k:
                    src, dst = np.array(k), first[b] + np.arange(len(k))
                    rows[torch.from_numpy(table[b, dst // page]).long().cuda(), torch.from_numpy(dst % page).cuda()] = \
                        old[torch.from_numpy(table[b, src // page]).long().cuda(), torch.from_numpy(src % page).cuda()]
            assert torch.equal(t, want)


def test_compact_refusals_on_the_device():
    for c, buffers, _ in caches(16, 8, 3):
        before = [t.clone() for t in buffers]
        table = ints([[0, 1, 2], [3, 4, 5]])
        for first, keep, n, bad in (
                ([5, 0], [[7, 6], [1, 2]], [2, 0], None), ([5, 0], [[4, 6], [1, 2]], [2, 0], None), ([5, 0], [[7, 7], [1, 2]], [2, 0], None),
                ([5, 0], [[7, 48], [1, 2]], [2, 0], None), ([5, 0], [[7, 9], [1, 2]], [3, 0], None), ([5, 0], [[7, 9], [1, 2]], [-1, 0], None),
                ([-1, 0], [[7, 9], [1, 2]], [2, 0], None), ([5, 0], [[7, 20], [1, 2]], [2, 0], 8), ([5, 0], [[7, 20], [1, 2]], [2, 0], -1)):
            t = table.clone()
            if bad is not None:
                t[0, 1] = bad
            qvg.paged_compact(c, t, ints(first), ints(keep), ints(n))
            assert qvg.get_status() == BAD, (first, keep, n)
            assert all(torch.equal(x, y) for x, y in zip(buffers, before))
        qvg.paged_compact(c, table, ints([5, 1]), ints([[7, 6], [1, 3]]), ints([2, 2]))  # the other sequence moves
        assert qvg.get_status() == BAD
        for t, was in zip(buffers, before):
            rows, old = (t[3], was[3]) if isinstance(c, qvg.LatentKV) else (t[3].transpose(0, 1), was[3].transpose(0, 1))
            assert torch.equal(rows[2], old[3]) and torch.equal(rows[3:], old[3:]) and torch.equal(t[:3], was[:3])
        qvg.paged_compact(c, table, ints([0, 0]), torch.zeros(2, 0, dtype=torch.int32, device="cuda"), ints([0, 0]))


def test_beam_over_a_paged_cache():
    """A sequence forked in three, each with its own next tokens, attends as if
    each beam had been written alone: the copies on write keep them apart."""
    H, d, page, n = 2, 64, 16, 37
    cache = qvg.PagedKV(H, d, page, 20)
    b = Both(20, 4, 4, page)
    g = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda m: torch.randn(m, H, d, generator=g, device="cuda").bfloat16()  # noqa: E731
    k, v = rnd(n), rnd(n)
    slots, copies = b.reserve([n, 0, 0, 0])
    qvg.paged_append(cache, k, v, slots)
    b.fork([0, 0, 0], [1, 2, 3])
    nk, nv = rnd(12), rnd(12)
    slots, copies = b.reserve([3] * 4)
    qvg.pages_copy(cache, copies)
    qvg.paged_append(cache, nk, nv, slots)
    assert int((copies[:, 0] >= 0).sum()) == 3
    q = rnd(4)
    out, _ = qvg.paged_attention(cache, q, b.table, b.len, 1)
    for i in range(4):
        alone = qvg.PagedKV(H, d, page, 4)
        qvg.paged_append(alone, torch.cat((k, nk[3 * i:3 * i + 3])), torch.cat((v, nv[3 * i:3 * i + 3])), torch.arange(n + 3, device="cuda"))
        want, _ = qvg.paged_attention(alone, q[i:i + 1], ints([[0, 1, 2, 3]]), ints([n + 3]), 1)
        # (the split of the work follows the batch: fp32 sums in another order, then half a bf16 step each)
        assert (out[i].double() - want[0].double()).abs().max() <= 2.0 ** -7 * want.double().abs().max()
    assert qvg.get_status() == OK
