"""dt_page_plan on the GPU against the same bookkeeping with lists. Whole numbers: everything is equal."""
import random

import pytest
import torch

pytestmark = pytest.mark.gpu
I32 = torch.int32


def ints(x):
    return torch.tensor(x, dtype=I32, device="cuda")


class Pool:
    """The reference: tables, held pages and the stack of free ones, as lists."""

    def __init__(self, B, pages, width, page, seed=0, spare=0):
        self.B, self.pages, self.width, self.page = B, pages, width, page
        order = list(range(pages))
        random.Random(seed).shuffle(order)
        self.free = order + [-9] * spare
        self.count = pages - spare
        self.table = [[-1] * width for _ in range(B)]
        self.held = [0] * B

    def tensors(self):
        return dict(page_table=ints(self.table), held=ints(self.held), free_pages=ints(self.free),
                    free_count=ints([self.count]))

    def step(self, lens, grow, n=0, rows=0, depth=None, path=None):
        """-> (lens, cu_seqlens, slots, positions), the requests that were not served."""
        page = self.page
        ends = [max(x, 0) + (g if x >= 0 else 0) for x, g in zip(lens, grow)]
        want = [-(-e // page) for e in ends]
        counts = [(n or (g if x >= 0 else 0)) for x, g in zip(lens, grow)]
        starts = [0]
        for c in counts:
            starts.append(starts[-1] + max(c, 0))
        bad = []
        for b in range(self.B):
            g = grow[b] if lens[b] >= 0 else 0
            late = rows and starts[b + 1] > rows
            bad.append(g < 0 or (n and g > n) or ends[b] > self.width * page or late or
                       not 0 <= self.held[b] <= self.width or (lens[b] >= 0 and self.held[b] * page < lens[b]))
        for b in reversed(range(self.B)):
            if not bad[b]:
                for i in reversed(range(want[b], self.held[b])):
                    self.free[self.count] = self.table[b][i]
                    self.count += 1
        full = False
        for b in range(self.B):
            need = want[b] - self.held[b]
            if bad[b] or need <= 0:
                if not bad[b]:
                    self.held[b] = want[b]
                continue
            full = full or need > self.count
            if full:
                bad[b] = True
                continue
            for i in range(self.held[b], want[b]):
                self.count -= 1
                self.table[b][i] = self.free[self.count]
            self.held[b] = want[b]
        out_lens = [0 if bad[b] else ends[b] for b in range(self.B)]
        slots, positions = [-1] * rows, [0] * rows
        for b in range(self.B):
            if bad[b] or not rows:
                continue
            for i in range(starts[b + 1] - starts[b]):
                g = grow[b] if lens[b] >= 0 else 0
                j = i
                if path is not None:
                    j = next((j for j in range(g) if path[b][j] == i), g)
                if j < g:
                    at = max(lens[b], 0) + j
                    slots[starts[b] + i] = self.table[b][at // page] * page + at % page
                    positions[starts[b] + i] = at if depth is None else lens[b] + depth[b][i] - 1
        starts = [min(x, rows) for x in starts] if rows else starts
        return (out_lens, starts, slots, positions), bad


def check(dtlib, ref, state, lens, grow, n=0, rows=0, depth=None, path=None, status=None, ws=None):
    want, bad = ref.step(lens, grow, n, n * ref.B if n else rows, depth, path)
    ws = dtlib.new_workspace(dtlib.dt_page_plan_workspace_bytes(ref.B)) if ws is None else ws
    out = dtlib.dt_page_plan(ints(lens), ints(grow), page_size=ref.page, num_pages=ref.pages, n=n, rows=rows,
                             depth=None if depth is None else ints(depth), path=None if path is None else ints(path),
                             workspace=ws, **state)
    assert dtlib.dt_get_error(ws) == (status if status is not None else dtlib.Status.OK)
    assert out["lens"].tolist() == want[0]
    assert out["cu_seqlens"].tolist() == want[1]
    if n or rows:
        assert out["slots"].tolist() == want[2]
        assert out["positions"].tolist() == want[3]
    else:
        assert "slots" not in out
    assert state["page_table"].tolist() == ref.table
    assert state["held"].tolist() == ref.held
    assert state["free_count"].tolist() == [ref.count]
    assert state["free_pages"].tolist()[:ref.count] == ref.free[:ref.count]
    return out, bad


@pytest.mark.parametrize("page", [8, 16, 64, 256])
@pytest.mark.parametrize("B,n", [(1, 0), (1, 1), (3, 5), (64, 16), (130, 0), (1500, 2), (2048, 0)])
def test_steps_of_a_serving_loop(dtlib, B, n, page):
    """Prompts admitted; trees with their accepted paths, or single tokens; requests that end and others in their place;
    the stack whole again at the end."""
    r = random.Random(B * 100 + n)
    longest = 300 if B > 100 else 1000
    width = -(-(longest + 400) // page)
    ref = Pool(B, B * width + 3, width, page, seed=B)
    state = ref.tensors()
    lens = [0] * B
    grow = [r.choice([0, 1, 7, r.randint(1, longest)]) for _ in range(B)]
    check(dtlib, ref, state, lens, grow, rows=sum(grow) + 11)
    lens = grow
    for round_ in range(3):
        if n:
            depth = [[r.randint(1, n) for _ in range(n)] for _ in range(B)]
            live = [n if r.random() < 0.9 else 0 for _ in range(B)]
            check(dtlib, ref, state, lens, live, n=n, depth=depth)
            kept = [r.randint(0, x) for x in live]
            path = [sorted(r.sample(range(n), a)) + [-1] * (n - a) for a in kept]
            check(dtlib, ref, state, lens, kept, n=n, path=path)
            lens = [x + a for x, a in zip(lens, kept)]
        grow = [r.randint(0, 40) if r.random() < 0.5 else 0 for _ in range(B)]
        check(dtlib, ref, state, lens, grow, rows=sum(grow))
        lens = [x + g for x, g in zip(lens, grow)]
        ended = [r.random() < 0.2 for _ in range(B)]
        check(dtlib, ref, state, [-1 - r.randint(0, 5) if e else x for e, x in zip(ended, lens)],
              [r.randint(-5, 5) if e else 0 for e in ended])
        lens = [0 if e else x for e, x in zip(ended, lens)]
    check(dtlib, ref, state, [-1] * B, [0] * B)
    assert ref.count == ref.pages and sorted(ref.free) == list(range(ref.pages))


def test_many_rows_take_a_second_launch(dtlib):
    for n, B, grow in ((0, 3, [9000, 0, 4001]), (0, 1, [8193]), (64, 200, None)):
        ref = Pool(B, 2000, 200, 64)
        state = ref.tensors()
        if n:
            r = random.Random(3)
            check(dtlib, ref, state, [0] * B, [n] * B, n=n)
            kept = [r.randint(0, n) for _ in range(B)]
            path = [sorted(r.sample(range(n), a)) + [-1] * (n - a) for a in kept]
            check(dtlib, ref, state, [0] * B, kept, n=n, path=path)
        else:
            check(dtlib, ref, state, [0] * B, grow, rows=sum(grow) + 700)
            check(dtlib, ref, state, grow, [1] * B, n=1)


@pytest.mark.parametrize("B,n", [(256, 1), (257, 1), (48, 16), (769, 1), (511, 1), (512, 1), (513, 1), (12, 64), (13, 64)])
def test_around_the_sizes_of_a_block(dtlib, B, n):
    """Requests and rows about what 256 threads take, of trees, of their accepted paths and of prompts with as many rows."""
    r = random.Random(B)
    ref = Pool(B, B * 12, 12, 16)
    state = ref.tensors()
    lens = [r.randint(0, 90) for _ in range(B)]
    check(dtlib, ref, state, [0] * B, lens, rows=sum(lens))
    check(dtlib, ref, state, lens, [n] * B, n=n, depth=[[r.randint(1, n) for _ in range(n)] for _ in range(B)])
    kept = [r.randint(0, n) for _ in range(B)]
    check(dtlib, ref, state, lens, kept, n=n, path=[sorted(r.sample(range(n), a)) + [-1] * (n - a) for a in kept])
    lens = [x + a for x, a in zip(lens, kept)]
    grow = [B * n // B if b else B * n - (B - 1) * (B * n // B) for b in range(B)]
    check(dtlib, ref, state, lens, [min(g, 30) for g in grow], rows=B * n)
    check(dtlib, ref, state, [-1 if b % 2 else x + min(g, 30) for b, (x, g) in enumerate(zip(lens, grow))], [0] * B)


def test_a_pool_that_runs_out(dtlib):
    ref = Pool(5, 10, 20, 16)
    state = ref.tensors()
    _, bad = check(dtlib, ref, state, [0] * 5, [64, 16, 100, 0, 16], rows=196, status=dtlib.Status.NO_PAGES)
    assert bad == [False, False, True, False, True]  # what comes behind the first that does not fit gets none
    # what others give back in the same step serves it
    _, bad = check(dtlib, ref, state, [-1, 16, 0, 0, 0], [0, 3, 100, 0, 16], rows=119)
    assert not any(bad)
    check(dtlib, ref, state, [0, 19, 100, 0, 16], [0, 13, 12, 0, 0], n=13)


def test_pages_given_and_taken_in_one_step_from_an_empty_stack(dtlib):
    ref = Pool(4, 8, 8, 8)
    state = ref.tensors()
    check(dtlib, ref, state, [0] * 4, [32, 32, 0, 0], rows=64)
    assert ref.count == 0
    check(dtlib, ref, state, [-1, 9, 0, 0], [0, 0, 30, 9], rows=39)
    assert ref.count == 0


def test_what_cannot_be_is_reported_and_left_out(dtlib):
    bad = dtlib.Status.INVALID_ARG
    for lens, grow, n in (([5, 5, 5], [3, -1, 2], 0),          # grows by less than nothing
                          ([5, 5, 5], [3, 4, 2], 3),           # more tokens than rows
                          ([5, 5, 5], [3, 8 * 16 - 4, 2], 0),  # more than its table holds
                          ([5, 2 ** 31 - 1, 5], [3, 2 ** 31 - 1, 3], 0),
                          ([5, 20, 5], [3, 1, 1], 3)):         # keeps more than it holds
        ref = Pool(3, 40, 8, 16)
        state = ref.tensors()
        check(dtlib, ref, state, [0] * 3, [5] * 3, rows=15)
        # the packed rows behind such a request may lie behind the rows that there are
        rows = 0 if n else sum(max(g, 0) for g in grow if g < 2 ** 20)
        _, out = check(dtlib, ref, state, lens, grow, n=n, rows=rows, status=bad)
        assert out[1] and not out[0]
    ref = Pool(3, 40, 8, 16)
    check(dtlib, ref, ref.tensors(), [0] * 3, [5, 6, 7], rows=12, status=bad)  # the last request's rows are not all there
    for held in (-1, 9, 2 ** 31 - 1):
        ref = Pool(3, 40, 8, 16)
        ref.held[1] = held
        check(dtlib, ref, ref.tensors(), [0] * 3, [5, 6, 7], rows=18, status=bad)
        ref.held[1] = held
        check(dtlib, ref, ref.tensors(), [5, -1, 0], [0, 0, 0], status=bad)


@pytest.mark.parametrize("count", [-1, 41, 39, 2 ** 31 - 1, -2 ** 31])
def test_a_pool_that_contradicts_itself_moves_nothing(dtlib, count):
    """39 free pages and two given back into a pool of 40; other counts are no counts at all."""
    ref = Pool(3, 40, 8, 16)
    state = ref.tensors()
    ws = dtlib.new_workspace(dtlib.dt_page_plan_workspace_bytes(3))
    check(dtlib, ref, state, [0] * 3, [20, 20, 20], rows=60)
    state["free_count"].fill_(count)
    before = {k: v.clone() for k, v in state.items()}
    out = dtlib.dt_page_plan(ints([-1, 20, 20]), ints([0, 2, 30]), page_size=16, num_pages=40, rows=32, workspace=ws,
                             **state)
    assert dtlib.dt_get_error(ws) == dtlib.Status.INVALID_ARG
    assert all(torch.equal(before[k], state[k]) for k in state)
    assert out["lens"].tolist() == [0, 22, 0]  # who needs no page has its rows
    assert (out["slots"][:2] >= 0).all() and (out["slots"][2:] == -1).all()


def test_pages_outside_the_pool_that_move_are_reported(dtlib):
    """An entry that is no page, given back by a request or taken from the stack: it moves as it is, and the status says so,
    with rows and without, of one block and of many."""
    for B, rows in ((3, 0), (3, 90), (300, 0), (300, 9000)):
        for page in (-1, 40 * B, 2 ** 31 - 1, -2 ** 31):
            ref = Pool(B, 40 * B, 500, 16)
            state = ref.tensors()
            check(dtlib, ref, state, [0] * B, [30] * B, rows=30 * B)
            # given back
            state["page_table"][1, 1] = ref.table[1][1] = page
            lens = [30, -1] + [30] * (B - 2)
            check(dtlib, ref, state, lens, [0] * B, status=dtlib.Status.INVALID_ARG)
            # taken: it lies on top of the stack, under the first page of request 1
            grow = [0, 30] + [0] * (B - 2)
            lens[1] = 0
            assert ref.free[ref.count - 2] == page
            ws = dtlib.new_workspace(dtlib.dt_page_plan_workspace_bytes(B))
            want, bad = ref.step(lens, grow, rows=rows)
            out = dtlib.dt_page_plan(ints(lens), ints(grow), page_size=16, num_pages=40 * B, rows=rows, workspace=ws, **state)
            assert dtlib.dt_get_error(ws) == dtlib.Status.INVALID_ARG and not any(bad)
            assert out["lens"].tolist() == want[0] and state["held"].tolist() == ref.held
            assert state["page_table"].tolist() == ref.table and state["free_count"].tolist() == [ref.count]
            if rows:  # the page's rows are no tokens, the others' are
                assert out["slots"].tolist() == [-1 if i >= 16 and i < 30 else x for i, x in enumerate(want[2])]
            # nothing that moves is outside: nothing is reported
            lens[1] = 30
            check(dtlib, ref, state, [-1 if b == 0 else x for b, x in enumerate(lens)], [0] * B)


def test_without_a_pool_the_table_is_read(dtlib):
    table = ints([[7, 3, -1], [9, 1, 2]])
    ws = dtlib.new_workspace(dtlib.dt_page_plan_workspace_bytes(2))
    out = dtlib.dt_page_plan(ints([15, 40]), ints([3, 2]), table, 16, 10, rows=6, workspace=ws)
    assert out["slots"].tolist() == [7 * 16 + 15, 3 * 16, 3 * 16 + 1, 2 * 16 + 8, 2 * 16 + 9, -1]
    assert out["positions"].tolist() == [15, 16, 17, 40, 41, 0] and out["cu_seqlens"].tolist() == [0, 3, 5]
    assert dtlib.dt_get_error(ws) == dtlib.Status.OK
    assert table.tolist() == [[7, 3, -1], [9, 1, 2]]
    out = dtlib.dt_page_plan(ints([31, 40]), ints([2, 1]), table, 16, 10, n=2, workspace=ws)  # a page that is none
    assert out["slots"].tolist() == [3 * 16 + 15, -1, 2 * 16 + 8, -1]
    assert dtlib.dt_get_error(ws) == dtlib.Status.INVALID_ARG
    out = dtlib.dt_page_plan(ints([31, 40]), ints([1, 1]), table, 16, 2, n=1, workspace=ws)  # pages past the pool
    assert out["slots"].tolist() == [-1, -1] and dtlib.dt_get_error(ws) == dtlib.Status.INVALID_ARG


def test_paths_of_any_content_stay_in_bounds(dtlib):
    table = ints([[4, 5]])
    for path in ([[2, 2, 0, 9]], [[-1, -7, 2 ** 31 - 1, 1]]):
        out = dtlib.dt_page_plan(ints([3]), ints([4]), table, 16, 10, n=4, path=ints(path))
        want = [next((64 + 3 + j for j in range(4) if path[0][j] == i), -1) for i in range(4)]
        assert out["slots"].tolist() == want


@pytest.mark.parametrize("n,grow", [(4, 5), (4, 1000), (4, 2 ** 31 - 1), (1, 2), (64, 65)])
def test_a_path_of_a_request_that_grows_by_too_much_is_not_read(dtlib, n, grow):
    """More accepted nodes than the tree has: reported, no tokens, the neighbours as they are. The path's rows lie inside a
    larger array, whose other entries would name every node; the last request's row is the array's last."""
    B, page = 3, 16
    around = torch.arange(5000 + B * n, dtype=I32, device="cuda") % n
    path = around[-B * n:].view(B, n)
    for which in range(B):
        ref = Pool(B, 40, 20, page)
        state = ref.tensors()
        check(dtlib, ref, state, [0] * B, [40] * B, rows=40 * B)
        kept = [min(2, n)] * B
        kept[which] = grow
        ws = dtlib.new_workspace(dtlib.dt_page_plan_workspace_bytes(B))
        want, bad = ref.step([30] * B, kept, n, n * B, path=path.tolist())
        out = dtlib.dt_page_plan(ints([30] * B), ints(kept), page_size=page, num_pages=40, n=n, path=path, workspace=ws,
                                 **state)
        assert bad == [b == which for b in range(B)]
        assert dtlib.dt_get_error(ws) == dtlib.Status.INVALID_ARG
        assert [out[k].tolist() for k in ("lens", "cu_seqlens", "slots", "positions")] == list(want)
        assert (out["slots"].view(B, n)[which] == -1).all() and (out["positions"].view(B, n)[which] == 0).all()
        assert state["page_table"].tolist() == ref.table and state["held"].tolist() == ref.held


def test_some_outputs_alone(dtlib):
    table, ws = ints([[7, 3, -1], [9, 1, 2]]), dtlib.new_workspace(dtlib.dt_page_plan_workspace_bytes(2))
    for out in (dict(lens=ints([0, 0])), dict(cu_seqlens=ints([0, 0, 0])), {}, dict(slots=ints([0] * 5), positions=ints([0] * 5))):
        got = dtlib.dt_page_plan(ints([15, 40]), ints([3, 2]), table, 16, 10, out=out, workspace=ws)
        assert got is out
        want = dict(lens=[18, 42], cu_seqlens=[0, 3, 5], slots=[127, 48, 49, 40, 41], positions=[15, 16, 17, 40, 41])
        assert all(out[k].tolist() == want[k] for k in out)


@pytest.mark.parametrize("pool", [True, False])
def test_an_empty_batch_has_a_first_row(dtlib, pool):
    """cu_seqlens has one entry, 0, also without requests and rows, as a call or in a graph; the pool stays as it is."""
    state = dict(page_table=ints([[]] * 0).view(0, 4))
    if pool:
        state.update(held=ints([]), free_pages=ints([3, 1, 2, 0, -9]), free_count=ints([4]))
    before = {k: v.clone() for k, v in state.items()}
    none = ints([])
    call = lambda **kw: dtlib.dt_page_plan(none, none, page_size=16, num_pages=5, **state, **kw)
    for n in (0, 3):
        out = dict(lens=ints([]), cu_seqlens=ints([77, 78])[:1])
        call(n=n, out=out)
        assert out["cu_seqlens"].tolist() == [0]
        assert call(n=n)["cu_seqlens"].tolist() == [0]
        g, out = torch.cuda.CUDAGraph(), dict(cu_seqlens=ints([77]))
        ws = dtlib.new_workspace(256)
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            call(n=n, out=out, workspace=ws)
        out["cu_seqlens"].fill_(5)
        g.replay()
        assert out["cu_seqlens"].tolist() == [0]
    rows = dict(cu_seqlens=ints([77]), slots=ints([5] * 9), positions=ints([5] * 9))
    call(out=rows)
    assert rows["cu_seqlens"].tolist() == [0] and rows["slots"].tolist() == [-1] * 9
    assert all(torch.equal(before[k], state[k]) for k in state)


def test_captured_and_replayed(dtlib):
    """A step of a loop as a graph: each replay takes the pages of one more token per request."""
    ref = Pool(3, 40, 10, 8)
    state = ref.tensors()
    check(dtlib, ref, state, [0] * 3, [7, 8, 9], rows=24)
    lens, grow = ints([7, 8, 9]), ints([1, 1, 1])
    out = dict(lens=ints([0] * 3), slots=ints([0] * 3), positions=ints([0] * 3))
    ws = dtlib.new_workspace(dtlib.dt_page_plan_workspace_bytes(3))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dtlib.dt_page_plan(lens, grow, page_size=8, num_pages=40, n=1, out=out, workspace=ws, **state)
        lens.copy_(out["lens"])
    for i in range(20):
        want, _ = ref.step([7 + i, 8 + i, 9 + i], [1] * 3, 1, 3)
        g.replay()
        assert (out["lens"].tolist(), out["slots"].tolist(), out["positions"].tolist()) == (want[0], want[2], want[3])
    assert state["page_table"].tolist() == ref.table and state["free_count"].tolist() == [ref.count]


@pytest.mark.parametrize("pool", [True, False])
@pytest.mark.parametrize("over", ["lens", "grow"])
def test_lengths_in_the_place_of_the_old_ones(dtlib, over, pool):
    """out lens is lens, or grow, themselves: of a plan by one block and by many."""
    for B, most in ((3, 20), (300, 900)):
        r = random.Random(B)
        lens, grow = [r.randint(0, 40) for _ in range(B)], [r.randint(0, most) for _ in range(B)]
        ref = Pool(B, B * 60, 60, 16)
        state = ref.tensors()
        check(dtlib, ref, state, [0] * B, lens, rows=sum(lens))
        if pool:
            want, _ = ref.step(lens, grow, rows=sum(grow) + 5)
        else:
            check(dtlib, ref, state, lens, grow, rows=sum(grow) + 5)
            want, _ = ref.step(lens, grow, rows=sum(grow) + 5)
        old = dict(lens=ints(lens), grow=ints(grow))
        out = dict(lens=old[over], cu_seqlens=ints([0] * (B + 1)), slots=ints([0] * (sum(grow) + 5)),
                   positions=ints([0] * (sum(grow) + 5)))
        given = state if pool else dict(page_table=state["page_table"])
        dtlib.dt_page_plan(old["lens"], old["grow"], page_size=16, num_pages=ref.pages, out=out, **given)
        got = [out[k].tolist() for k in ("lens", "cu_seqlens", "slots", "positions")]
        assert got == list(want)


def test_refuses(dtlib):
    table, lens = ints([[7, 3, -1], [9, 1, 2]]), ints([1, 2])
    held, free, count = ints([1, 1]), ints([0] * 10), ints([0])
    call = lambda **kw: dtlib.dt_page_plan(**{**dict(lens=lens, grow=lens, page_table=table, page_size=16, num_pages=10), **kw})
    call(n=2)
    for bad in (dict(held=held), dict(held=held, free_pages=free), dict(page_size=0),
                dict(n=1, depth=ints([[1], [1]]), path=ints([[1], [1]])), dict(n=-1), dict(page_size=24), dict(page_size=512),
                dict(num_pages=2 ** 28)):
        with pytest.raises(dtlib.DTError):
            call(**bad)
    for bad in (dict(grow=ints([1])), dict(depth=ints([[1], [1]])), dict(page_table=table[:1]), dict(n=2, depth=ints([[1], [1]])), dict(
            held=held, free_pages=free[:9], free_count=count), dict(held=held, free_pages=free, free_count=ints([1, 2])),
            dict(n=2, out=dict(slots=ints([0] * 3), positions=ints([0] * 3))), dict(page_table=table.t())):
        with pytest.raises(ValueError):
            call(**bad)
    for bad in (dict(grow=lens.long()), dict(lens=lens.cpu()), dict(grow=lens.cpu()), dict(page_table=table.float())):
        with pytest.raises(TypeError):
            call(**bad)
