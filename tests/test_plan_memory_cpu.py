"""A plan that does not fit the host's memory is an error, not an abort: no exception leaves the C ABI."""
import subprocess
import sys

from paged_top_sparse_gb300 import build

CHILD = """
import resource
from paged_top_sparse_gb300 import binding as B
B.lib()
plan = lambda q: B.Plan([q], [0], 64, 64, 64, 1, q // 128, q // 128)
plan(1 << 17)
used = int(open("/proc/self/statm").read().split()[0]) * resource.getpagesize()
for room in (8, 24, 60, 100, 150, 200):  # MiB: the plan fails in one allocation after another
    resource.setrlimit(resource.RLIMIT_AS, (used + (room << 20), resource.RLIM_INFINITY))
    try:
        plan(1 << 20)
        print("planned")
    except B.SpsError as e:
        assert e.status == 1 and "memory" in str(e), e
        print("refused")
resource.setrlimit(resource.RLIMIT_AS, (resource.RLIM_INFINITY, resource.RLIM_INFINITY))
plan(1 << 17)
print("ok")
"""


def test_a_plan_without_memory_is_refused():
    build.build()
    r = subprocess.run([sys.executable, "-c", CHILD], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    lines = r.stdout.split()
    assert lines[-1] == "ok" and lines[0] == "refused", lines
