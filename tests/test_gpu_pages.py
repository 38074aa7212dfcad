"""Block tables, slots and positions of a step on the GPU against the oracle, number by number."""
import numpy as np
import pytest

import bit_unstructured_sparse_amd as bsp
from oracle import step

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    return torch.device("cuda:0")


def _state(rng, B, page, most, width, spare, dev):
    """Sequences of up to `most` tokens, their pages in any order, `spare` free ones; (pages on the GPU, oracle)."""
    lens = rng.integers(0, most + 1, B) if B else np.zeros(0, int)
    held = -(-lens // page)
    order = rng.permutation(int(held.sum()) + spare).astype(np.int32)
    table = np.full((B, width), 7, np.int32)
    at = 0
    for b in range(B):
        table[b, :held[b]] = order[at:at + held[b]]
        at += held[b]
    free = np.full(2 + order.size, -1, np.int32)
    free[0], free[1], free[2:2 + spare] = spare, 0, order[at:]
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.int32)).to(dev)
    pages = bsp.KVPages(t(table), t(lens), t(held), t(free), page)
    return pages, step.Pages(table, lens, held, order[at:], page)


def _compare(pages, out, ref, want, rows):
    slots, positions, sequences, q_start, kv_lens = want
    assert out.q_start.tolist() == q_start
    assert out.kv_lens.tolist() == kv_lens
    assert out.sequences.tolist() == sequences
    assert out.positions.tolist() == positions
    assert out.slots.tolist() == slots
    assert pages.lens.tolist() == ref.lens and pages.held.tolist() == ref.held
    free = pages.free.tolist()
    assert free[0] == len(ref.free) and free[1] == 0 and free[2:2 + len(ref.free)] == ref.free
    table = pages.block_table.tolist()
    for b, h in enumerate(ref.held):
        assert table[b][:h] == ref.table[b][:h]


def _i32(a, dev):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).to(dev)


@pytest.mark.parametrize("B", [1, 2, 31, 255, 256, 257, 700])
@pytest.mark.parametrize("page,most,spare", [(16, 100, 4096), (16, 300, 40), (64, 1000, 0), (4096, 9000, 50)])
def test_steps_one_after_the_other(B, page, most, spare, dev):
    rng = np.random.default_rng(B * 13 + page + spare)
    width = -(-(most + 80) // page)
    pages, ref = _state(rng, B, page, most, width, spare, dev)
    for k in range(6):
        # drafts kept in part, requests that end, prompts, nothing at all
        lens = np.array(ref.lens)
        keep = np.maximum(lens - rng.integers(0, 9, B), 0)
        keep = np.where(rng.random(B) < 0.15, 0, keep)
        new = np.where(rng.random(B) < 0.2, 0, rng.integers(0, 20, B))
        new = np.where(keep == 0, rng.integers(0, most + 1, B), new)
        rows = int(new.sum()) + int(rng.integers(0, 9)) - (3 if k == 4 else 0)
        rows = max(rows, 0)
        masks = rng.integers(0, 2 ** 63, rows, dtype=np.int64) if k % 2 else None
        use = None if k == 2 else keep
        out = bsp.kv_step(pages, None if use is None else _i32(use, dev), _i32(new, dev), rows,
                          tree_mask=None if masks is None else torch.from_numpy(masks).to(dev))
        torch.cuda.synchronize()
        want = ref.step(use, new, rows, None if masks is None else masks.view(np.uint64))
        _compare(pages, out, ref, want, rows)
        owned = [p for b, h in enumerate(ref.held) for p in ref.table[b][:h]] + ref.free
        assert sorted(owned) == list(range(len(owned))), "a page is lost or held twice"


@pytest.mark.parametrize("spare", [60, 10, 0])
def test_a_step_and_its_undoing(spare, dev):
    rng = np.random.default_rng(9)
    pages, ref = _state(rng, 90, 16, 200, 30, spare, dev)
    before = [t.clone() for t in (pages.block_table, pages.lens, pages.held, pages.free)]
    lens = np.array(ref.lens)
    keep = np.where(np.arange(90) % 7 == 3, 0, lens)
    new = np.where(np.arange(90) % 7 == 3, rng.integers(0, 100, 90), rng.integers(0, 30, 90))
    out = bsp.kv_step(pages, _i32(keep, dev), _i32(new, dev), int(new.sum()))
    assert (out.slots < 0).any() == (spare < 60)      # some wait, for want of pages
    bsp.kv_step(pages, _i32(keep, dev), _i32(lens - keep, dev), int((lens - keep).sum()))
    for a, b in zip(before, (pages.block_table, pages.lens, pages.held, pages.free)):
        if a.dim() == 2:      # entries past the held ones mean nothing
            inside = torch.arange(a.shape[1], device=dev)[None, :] < before[2][:, None]
            a, b = a[inside], b[inside]
        assert torch.equal(a, b)


def test_waiting(dev):
    # pool of 2 pages; sequence 0 takes 2, 1 needs none, 2 must wait and so must 3, which 4 gives back too late for
    P = 16
    t = lambda a: _i32(np.array(a), dev)
    pages = bsp.KVPages(t([[0, 0, 0]] * 5), t([0, 5, 16, 0, 16]), t([0, 1, 1, 0, 1]), t([2, 0, 8, 9]), P)
    out = bsp.kv_step(pages, None, t([17, 11, 1, 1, 0]), 40)
    assert out.kv_lens.tolist() == [17, 16, 0, 0, 16]
    assert pages.lens.tolist() == [17, 16, 16, 0, 16] and pages.held.tolist() == [2, 1, 1, 0, 1]
    assert out.slots[:17].tolist() == [9 * 16 + i for i in range(16)] + [8 * 16]
    assert (out.slots[28:30] == -1).all() and out.sequences[28:32].tolist() == [2, 3, -1, -1]
    assert out.positions[28:31].tolist() == [16, 0, 0]
    # the page of sequence 4 lets sequence 2 go on, not 3
    out = bsp.kv_step(pages, t([17, 16, 16, 0, 0]), t([0, 0, 1, 1, 0]), 2)
    assert out.kv_lens.tolist() == [17, 16, 17, 0, 0] and pages.held.tolist() == [2, 1, 2, 0, 0]
    # rows past the call's, pages past the table
    out = bsp.kv_step(pages, None, t([1, 0, 0, 4, 0]), 3)
    assert out.kv_lens.tolist() == [18, 16, 17, 0, 0] and out.q_start.tolist() == [0, 1, 1, 1, 3, 3]
    out = bsp.kv_step(pages, None, t([60, 0, 0, 0, 0]), 60)
    assert out.kv_lens.tolist()[0] == 0 and pages.lens.tolist()[0] == 18 and (out.slots == -1).all()


def test_values_that_cannot_be_touch_nothing_outside(dev):
    t = lambda a: _i32(np.array(a), dev)
    big = 2 ** 31 - 1
    guard = torch.full((64,), 77, dtype=torch.int32, device=dev)
    table, lens, held, free = guard[8:16].view(2, 4), guard[20:22], guard[24:26], guard[30:36]
    pages = bsp.KVPages(table, lens, held, free, 16)
    for values in (big, -big - 1, 1000, -1):
        for n in (lens, held, table, free):
            n.fill_(values)
        free[1] = 0
        for keep in (None, t([big, -5])):
            for new in ([big, big], [-3, 1], [0, 40]):
                out = bsp.kv_step(pages, keep, t(new), 7)
                torch.cuda.synchronize()
                assert int(pages.free[1]) == 0 and 0 <= int(free[0]) <= 4
                assert (out.kv_lens >= 0).all() and (out.kv_lens <= 64).all()
                assert 0 <= int(out.q_start.min()) and int(out.q_start.max()) <= 7
    outside = torch.ones(64, dtype=torch.bool, device=dev)
    for a, b in ((8, 16), (20, 22), (24, 26), (30, 36)):
        outside[a:b] = False
    assert (guard[outside] == 77).all()


def test_many_rows_and_most_sequences(dev):
    rng = np.random.default_rng(12)
    # the most sequences a call takes
    pages, ref = _state(rng, bsp.PAGES_MAX_SEQUENCES, 16, 40, 8, 3000, dev)
    new = rng.integers(0, 9, bsp.PAGES_MAX_SEQUENCES)
    rows = int(new.sum())
    out = bsp.kv_step(pages, None, _i32(new, dev), rows)
    _compare(pages, out, ref, ref.step(None, new, rows), rows)
    # one prompt over many workgroups
    pages, ref = _state(rng, 3, 128, 1000, 2000, 2000, dev)
    new = np.array([1, 200001, 5])
    out = bsp.kv_step(pages, None, _i32(new, dev), 200010)
    _compare(pages, out, ref, ref.step(None, new, 200010), 200010)


def test_no_sequences_and_no_rows(dev):
    pages = bsp.new_kv_pages(0, 4, 10, 16, device=dev)
    none = torch.empty(0, dtype=torch.int32, device=dev)
    out = bsp.kv_step(pages, None, none, 3)
    assert out.slots.tolist() == [-1] * 3 and out.sequences.tolist() == [-1] * 3 and out.q_start.tolist() == [0]
    pages = bsp.new_kv_pages(2, 4, 10, 16, device=dev)
    out = bsp.kv_step(pages, None, _i32([0, 0], dev), 0)
    assert out.q_start.tolist() == [0, 0, 0] and pages.free.tolist()[:2] == [10, 0]


def test_a_captured_step_replayed(dev):
    # the state moves on with every replay, as an eager twin's does; on a side stream too
    rng = np.random.default_rng(14)
    pages, ref = _state(rng, 40, 16, 100, 40, 200, dev)
    twin = bsp.KVPages(*(t.clone() for t in (pages.block_table, pages.lens, pages.held, pages.free)), 16)
    keep, new = _i32(ref.lens, dev), _i32(rng.integers(0, 9, 40), dev)
    rows = 400
    i32 = torch.int32
    out = bsp.KVStep(*(torch.zeros(n, dtype=t, device=dev) for n, t in
                       ((rows, torch.int64), (rows, i32), (rows, i32), (41, i32), (40, i32))))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bsp.kv_step(pages, keep, new, rows, out=out)
    side = torch.cuda.Stream()
    for k in range(4):
        keep.copy_((twin.lens - 2).clamp(min=0))
        new.copy_(_i32(rng.integers(0, 9, 40), dev))
        graph.replay()
        side.wait_stream(torch.cuda.current_stream())
        eager = bsp.kv_step(twin, keep, new, rows, stream=side)
        torch.cuda.synchronize()
        for a, b in zip(out, eager):
            assert torch.equal(a, b)
        for a, b in ((pages.lens, twin.lens), (pages.held, twin.held), (pages.free, twin.free),
                     (pages.block_table, twin.block_table)):
            assert torch.equal(a, b)


def test_two_states_at_once(dev):
    rng = np.random.default_rng(15)
    both = [_state(rng, 300, 16, 200, 30, 500, dev) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs, news = [], [rng.integers(0, 40, 300) for _ in range(2)]
    new = [_i32(n, dev) for n in news]
    torch.cuda.synchronize()
    for (pages, _), s, n, d in zip(both, streams, news, new):
        outs.append(bsp.kv_step(pages, None, d, int(n.sum()), stream=s))
    torch.cuda.synchronize()
    for (pages, ref), n, out in zip(both, news, outs):
        _compare(pages, out, ref, ref.step(None, n, int(n.sum())), int(n.sum()))
