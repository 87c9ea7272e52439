"""The work split of the full attention, from the tables that a plan uploads: every page of every tile
on one block, and the slots, merges and room that the kernels rely on.  No GPU is needed."""
import ctypes

import numpy as np
import pytest

from paged_top_sparse_gb300 import binding as B
from paged_top_sparse_gb300 import build

PIECE = np.dtype([(n, np.int32) for n in ("req", "vg", "tile", "page0", "page1", "q_len", "ctx", "flat0")])
HEAD = np.dtype([("first", PIECE), ("count", np.int32), ("next", np.int32), ("pad", np.int32, 2)])
MERGE = np.dtype([(n, np.int32) for n in ("req", "vg", "tile", "cta0", "cta1", "q_len", "flat0", "pad")])


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


class Tables:
    """What the plan of a batch uploads for the attention."""

    def __init__(self, q_lens, ctx, H, G):
        pages = max((c + q - 1) // 128 + 1 for q, c in zip(q_lens, ctx) if q)
        self.plan = B.Plan(q_lens, ctx, H, G, 64, 1, pages, pages)
        L = B.lib()
        L.sps_internal_attention_tables.restype = ctypes.c_void_p
        info = (ctypes.c_int64 * 8)()
        base = L.sps_internal_attention_tables(self.plan.handle, info)
        (self.off_heads, self.off_pieces, self.off_merges, self.end, self.ctas, self.slot_rows,
         self.num_merges, self.merge_cap) = info
        raw = np.ctypeslib.as_array(ctypes.cast(base, ctypes.POINTER(ctypes.c_uint8)), (self.end,))
        assert self.off_heads == 0 and self.off_merges >= self.ctas * HEAD.itemsize
        assert self.off_pieces >= self.off_merges + self.ctas * MERGE.itemsize
        self.heads = raw[:self.ctas * HEAD.itemsize].view(HEAD)
        self.merges = raw[self.off_merges:][:self.ctas * MERGE.itemsize].view(MERGE)
        self.pieces = raw[self.off_pieces:self.end].view(PIECE)  # with the room behind them

    def blocks(self):
        """Each block's pieces in turn."""
        out, at = [], 0
        for h in self.heads:
            run = []
            if h["count"]:
                assert h["next"] == at  # neighbours in the table, none shared
                run = [h["first"]] + list(self.pieces[at:at + h["count"] - 1])
                at += h["count"] - 1
            out.append(run)
        assert at <= len(self.pieces)
        return out


def _check(q_lens, ctx, H, G):
    t = Tables(q_lens, ctx, H, G)
    hg = H // G
    HB = min(hg, 128)
    TB, per_group = 128 // HB, -(-hg // HB)
    flat = np.concatenate([[0], np.cumsum(q_lens)])
    tiles = {}
    for b, (q, c) in enumerate(zip(q_lens, ctx)):
        for v in range(G * per_group):
            for i in range(-(-q // (2 * TB))):
                tiles[b, v, i] = (c + min((i + 1) * 2 * TB, q) - 1) // 128 + 1
    assert t.slot_rows == (256 if max(q_lens) > TB else max(q_lens) * HB)
    parts, slots = {}, set()
    for cta, run in enumerate(t.blocks()):
        for n, x in enumerate(run):
            key = (int(x["req"]), int(x["vg"]), int(x["tile"]))
            a, e = int(x["page0"]), int(x["page1"])
            assert 0 <= a < e <= tiles[key]
            assert (x["q_len"], x["ctx"], x["flat0"]) == (q_lens[key[0]], ctx[key[0]], flat[key[0]])
            parts.setdefault(key, []).append((cta, a, e))
            if (a, e) != (0, tiles[key]):
                # the kernels' slot of a partial result: by whether the piece begins its tile
                slot = 2 * cta + (0 if a else 1)
                assert slot not in slots
                slots.add(slot)
    assert parts.keys() == tiles.keys()
    cut = {}
    for key, p in parts.items():
        p.sort(key=lambda x: x[1])
        assert [x[1] for x in p] == [0] + [x[2] for x in p[:-1]] and p[-1][2] == tiles[key]
        if len(p) > 1:  # the merge walks neighbouring blocks
            assert [x[0] for x in p] == list(range(p[0][0], p[0][0] + len(p)))
            cut[key] = (p[0][0], p[-1][0])
    got = t.merges[:t.num_merges]
    assert {(int(m["req"]), int(m["vg"]), int(m["tile"])): (int(m["cta0"]), int(m["cta1"]))
            for m in got} == cut and len(cut) == t.num_merges
    for m in got:
        assert m["q_len"] == q_lens[m["req"]] and m["flat0"] == flat[m["req"]]
    # a captured call launches merge_cap of them over whatever plan was uploaded since
    assert t.num_merges <= t.merge_cap == min(t.ctas - 1, len(tiles))
    assert bool((t.merges["req"][t.num_merges:] == -1).all())
    return t


@pytest.mark.parametrize("q_lens,ctx,H,G", [
    ([1], [0], 1, 1), ([1], [(1 << 20) - 1], 8, 1), ([8192], [0], 32, 2), ([512] * 8, [32768] * 8, 32, 2),
    ([1] * 64, [32768 + 977 * i for i in range(64)], 32, 2), ([1] * 700, [100] * 700, 4, 2),
    ([3] * 152, [127] * 152, 1, 1), ([1, 0, 130, 7, 300, 1, 128, 1], [0, 5, 1000, 121, 0, 127, 128, 4000], 6, 2),
    ([40, 1], [20000, 30000], 160, 1), ([5000], [77], 33, 3), ([2000] + [1] * 100, [0] * 101, 4, 4),
])
def test_split_of_given_batches(q_lens, ctx, H, G):
    _check(q_lens, ctx, H, G)


@pytest.mark.parametrize("seed", range(8))
def test_split_of_random_batches(seed):
    rng = np.random.default_rng(seed)
    for _ in range(40):
        n = int(rng.choice([1, 2, 5, 20, 150, 400]))
        top_q = int(rng.choice([1, 3, 40, 600 if n < 100 else 40]))
        top_c = int(np.exp(rng.uniform(0, np.log(200000 if n < 30 else 5000))))
        q_lens = [int(x) for x in rng.integers(0 if rng.random() < 0.3 else 1, top_q + 1, n)]
        q_lens[0] = max(1, q_lens[0])
        ctx = [int(x) for x in rng.integers(0, top_c + 1, n)]
        if rng.random() < 0.3:
            ctx[int(rng.integers(n))] = 400000  # one long context beside the others
        G = int(rng.choice([1, 2, 3, 8]))
        _check(q_lens, ctx, G * int(rng.choice([1, 3, 4, 7, 16, 128, 130])), G)


def test_tables_lie_where_lengths_and_heads_say():
    """A captured call is replayed over the tables of plans with other contexts."""
    for q_lens, H, G in (([1] * 9, 16, 2), ([300, 1, 70], 8, 8)):
        want = None
        for ctx in ([0] * len(q_lens), [127] * len(q_lens), [50000 - 777 * i for i in range(len(q_lens))]):
            t = _check(q_lens, ctx, H, G)
            i = t.plan.info()
            got = (t.off_heads, t.off_pieces, t.off_merges, t.end, t.ctas, t.slot_rows, t.merge_cap,
                   i.off_status, i.off_tok_pos, i.off_tok_req, B.paged_attention_scratch(t.plan))
            assert want in (None, got)
            want = got
