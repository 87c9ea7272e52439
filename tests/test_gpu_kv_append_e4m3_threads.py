"""Host threads append into E4M3 caches of their own, with rotations of different size."""
import threading

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.mark.parametrize("D,rots", [(128, (32, 128)), (64, (64, 48))])
def test_rotations_of_different_size_on_threads(D, rots):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_top_sparse_gb300 import binding as B
    from paged_top_sparse_gb300 import build

    build.build()
    T, G, PAGES, ROUNDS = 9, 1, 1, 20000

    class Side:
        def __init__(self, rot):
            g = torch.Generator(device=DEV)
            g.manual_seed(rot)
            self.plan = B.Plan([T], [0], G, G, D, 1, PAGES, PAGES, kv_dtype="e4m3")
            self.ws = torch.zeros(self.plan.workspace_bytes, dtype=torch.uint8, device=DEV)
            B.sps_plan_upload(self.plan, self.ws)
            f = 1e4 ** (-torch.arange(rot // 2, dtype=torch.float64) * 2 / rot)
            self.rope = B.Rope(f.float().to(DEV))
            self.new = torch.randn((T, 2 * G, D), generator=g, device=DEV).bfloat16()
            self.pt = torch.zeros((1, PAGES), dtype=torch.int32, device=DEV)
            self.stream, self.codes = torch.cuda.Stream(), {}

        def caches(self):
            return [torch.zeros((PAGES, G, 128, D), dtype=torch.uint8, device=DEV) for _ in "kv"] + \
                [torch.zeros((PAGES, G), device=DEV) for _ in "kv"]

        def append(self, caches, stream):
            # straight to the library: what surrounds a call would keep the threads apart
            new, kv = self.new.data_ptr(), [c.data_ptr() for c in caches]
            args = (self.plan.handle, new, 2 * G * D, new + 2 * G * D, 2 * G * D, None, 1e-6, self.rope.ref,
                    self.pt.data_ptr(), *kv, self.ws.data_ptr(), stream.cuda_stream)
            call = B.lib().sps_kv_append_rope
            return lambda: call(*args)

        def loop(self, caches):
            call = self.append(caches, self.stream)
            for _ in range(ROUNDS):
                st = call()
                self.codes[st] = self.codes.get(st, 0) + 1

    sides = [Side(r) for r in rots]
    want, got = [s.caches() for s in sides], [s.caches() for s in sides]
    for s, w in zip(sides, want):
        assert s.append(w, torch.cuda.current_stream())() == 0
    torch.cuda.synchronize()
    threads = [threading.Thread(target=s.loop, args=(c,)) for s, c in zip(sides, got)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert [s.codes for s in sides] == [{0: ROUNDS}] * 2
    for s, w, c in zip(sides, want, got):
        assert B.sps_read_device_status(s.plan, s.ws) == 0
        assert all(torch.equal(x, y) for x, y in zip(w, c))
