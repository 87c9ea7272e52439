"""GPU checks of sps_page_tables: tables, slots and positions against a plain loop, batches of every size,
requests without new tokens, room behind the last token, exhausted lists and bad lengths, graph replay."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_top_sparse_gb300 import build

    build.build()


def plain(q, c, free, head, table, room):
    table, slots, pos, starts = table.copy(), np.full(room, -1, np.int64), np.zeros(room, np.int32), [0]
    t = 0
    for b, (n, ctx) in enumerate(zip(q, c)):
        for p in range(-(-ctx // 128), -(-(ctx + n) // 128)):
            table[b, p] = free[head]
            head += 1
        for i in range(n):
            pos[t] = ctx + i
            phys = table[b, (ctx + i) // 128]
            slots[t] = int(phys) * 128 + (ctx + i) % 128 if phys >= 0 else -1
            t += 1
        starts.append(t)
    return table, slots, pos, np.array(starts, np.int32), head


class Call:
    def __init__(self, q, c, width, num_free, head=0, extra=3, seed=0):
        from paged_top_sparse_gb300 import binding as B

        self.B, self.q, self.c = B, q, c
        rng = np.random.default_rng(seed)
        dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
        ids = rng.permutation(num_free + 100000).astype(np.int32)
        self.table = np.full((len(q), width), -7, np.int32)
        at = num_free
        for b, ctx in enumerate(c):
            n = max(0, min(width, -(-ctx // 128)))
            self.table[b, :n] = ids[at % 90000:at % 90000 + n]
            at += n
        self.free, self.head, self.room = ids[:num_free], head, max(0, sum(max(0, x) for x in q)) + extra
        self.d = dict(q_lens=dev(np.array(q, np.int32)), ctx_lens=dev(np.array(c, np.int32)),
                      free_pages=dev(self.free), free_state=dev(np.array([head, 0], np.int32)),
                      page_table=dev(self.table), slots=torch.full((self.room,), 99, dtype=torch.int64, device=DEV),
                      positions=torch.full((self.room,), 99, dtype=torch.int32, device=DEV),
                      starts=torch.full((len(q) + 1,), 99, dtype=torch.int32, device=DEV),
                      dev_status=torch.zeros(1, dtype=torch.int32, device=DEV))

    def run(self, **kw):
        self.B.sps_page_tables(**dict(self.d, **kw))
        torch.cuda.synchronize()
        return int(self.d["dev_status"])

    def check(self):
        table, slots, pos, starts, head = plain(self.q, self.c, self.free, self.head, self.table, self.room)
        got = {k: v.cpu().numpy() for k, v in self.d.items()}
        assert np.array_equal(got["page_table"], table)
        assert np.array_equal(got["slots"], slots) and np.array_equal(got["positions"], pos)
        assert np.array_equal(got["starts"], starts) and got["free_state"].tolist() == [head, 0]

    def check_untouched(self):
        got = {k: v.cpu().numpy() for k, v in self.d.items()}
        assert np.array_equal(got["page_table"], self.table) and got["free_state"].tolist() == [self.head, 0]
        assert (got["slots"] == -1).all() and (got["positions"] == 0).all() and (got["starts"] == 0).all()


@pytest.mark.parametrize("q,c", [
    ([1], [0]), ([1], [127]), ([1], [128]), ([0], [5]), ([0, 0], [0, 300]), ([128], [0]), ([129], [255]),
    ([1, 0, 130, 7, 300, 1, 128, 1], [0, 5, 1000, 121, 0, 127, 128, 4000]),
    ([1] * 64, [24576 + 257 * i for i in range(64)]),
])
def test_tables(q, c):
    call = Call(q, c, 400, 40, head=3)
    assert call.run() == 0
    call.check()


@pytest.mark.parametrize("batch,q_hi", [(1, 70000), (255, 3), (256, 900), (257, 400), (1000, 40), (5000, 2), (16384, 3)])
def test_batches_of_every_size(batch, q_hi):
    rng = np.random.default_rng(batch)
    q = rng.integers(0, q_hi + 1, batch).tolist()
    c = rng.integers(0, 2000, batch).tolist()
    call = Call(q, c, (2000 + q_hi) // 128 + 2, 200000, extra=700, seed=batch)
    assert call.run() == 0
    call.check()


def test_outputs_that_are_not_wanted():
    call = Call([5, 200], [100, 1], 8, 9)
    for name in ("slots", "positions", "starts", "dev_status"):
        one = Call([5, 200], [100, 1], 8, 9)
        one.run(**{name: None})
        call.run() if name == "slots" else None
        for k in one.d:
            if k != name:
                assert torch.equal(one.d[k], call.d[k]), (name, k)
    none = Call([5, 200], [100, 1], 8, 9)
    none.run(slots=None, positions=None, starts=None, dev_status=None)
    assert torch.equal(none.d["page_table"], call.d["page_table"])


def test_a_table_entry_that_is_missing_gives_no_slot():
    call = Call([3], [10], 4, 4)
    call.d["page_table"][0, 0] = -1
    call.table[0, 0] = -1
    assert call.run() == 0
    call.check()


@pytest.mark.parametrize("q,c,free,head,room,code", [
    ([300, 1], [0, 128], 4, 1, None, 5),   # four pages, three left
    ([300, 1], [0, 128], 4, 5, None, 5),   # a counter behind the list
    ([300, 1], [0, 128], 4, -1, None, 5),
    ([-1, 5], [4, 4], 9, 0, None, 6), ([1, 5], [4, -4], 9, 0, None, 6),
    ([1, 600], [4, 500], 9, 0, None, 6),   # behind the row of eight pages
    ([2147483647, 1], [2147483647, 1], 9, 0, 10, 6),
    ([9, 9], [4, 4], 9, 0, 17, 6),         # one token more than the maps hold
])
def test_refused_batches_take_nothing(q, c, free, head, room, code):
    call = Call([min(x, 1000) for x in q], [min(x, 1000) for x in c], 8, free, head)
    call.d["q_lens"].copy_(torch.tensor(q, dtype=torch.int32))
    call.d["ctx_lens"].copy_(torch.tensor(c, dtype=torch.int32))
    if room is not None:
        call.room = room
        call.d["slots"], call.d["positions"] = call.d["slots"][:room].clone(), call.d["positions"][:room].clone()
    assert call.run() == code
    call.check_untouched()
    # the first code stays; the next batch is served as if nothing had happened
    assert call.run() == code
    call.check_untouched()
    if code == 6:
        call.d["q_lens"].fill_(1)
        call.d["ctx_lens"].fill_(0)
        call.d["dev_status"].zero_()
        call.table[:] = -7
        call.d["page_table"].fill_(-7)
        call.q, call.c, call.head = [1, 1], [0, 0], 0
        call.d["free_state"].zero_()
        assert call.run() == 0
        call.check()


def test_captured_loop_takes_pages_as_the_contexts_grow():
    q, c = [1, 1, 2, 0], [126, 0, 250, 60]
    call = Call(q, c, 9, 30)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        call.B.sps_page_tables(**call.d, stream=s)
        call.d["ctx_lens"].add_(call.d["q_lens"])
    table, head, c = call.table, call.head, list(c)
    for _ in range(300):
        graph.replay()
        table, slots, pos, starts, head = plain(q, c, call.free, head, table, call.room)
        torch.cuda.synchronize()
        assert np.array_equal(call.d["page_table"].cpu().numpy(), table)
        assert np.array_equal(call.d["slots"].cpu().numpy(), slots)
        assert call.d["free_state"].tolist() == [head, 0]
        c = [a + n for a, n in zip(c, q)]
    assert int(call.d["dev_status"]) == 0
