"""How large a batch sparse_prefill_fwd_noalloc takes: its array holds what the forward reads, and
nothing of the tables that other operators' calls read from a plan's workspace.  (Like its sibling,
named to run behind the other test files.)"""
import pytest

torch = pytest.importorskip("torch")

from paged_top_sparse_gb300 import synth

pytestmark = pytest.mark.gpu


def test_the_largest_prompt_of_32_heads_fits():
    """12,084 tokens x 32 heads x top-16 fill the 48 MiB but for 0.5 KB: 8 bytes a selection, the
    tokens' and pages' metadata, the indexer's items, the buckets.  The partials of this call equal
    those of the forward with a workspace, bit for bit."""
    from paged_top_sparse_gb300 import binding as B
    from paged_top_sparse_gb300 import build
    from tests.gpu_helpers import DeviceRun

    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    w = synth.workload("custom", seed=31, q_lens=[12084], ctx_lens=[0], num_q_heads=32, num_kv_heads=2,
                       head_dim=128, top_k=16)
    run = DeviceRun(w, synth.make_tensors(w))
    run.indexer()
    run.topk()
    run.partial.zero_()
    run.forward()
    partial, lse = torch.zeros_like(run.partial), torch.full_like(run.lse, float("nan"))
    status = torch.zeros(1, dtype=torch.int32, device=run.dev)
    B.sparse_prefill_fwd_noalloc(run.plan, run.q, run.q_scale, run.k, run.v, None, None,
                                 run.page_table, run.idx, partial, lse, dev_status=status)
    torch.cuda.synchronize()
    assert run.status() == 0 and int(status.item()) == 0
    assert torch.equal(partial, run.partial) and torch.equal(lse, run.lse)
    assert bool((partial != 0).any())
