"""Host memory that runs out inside a call is an error code of its own, not a C++ exception through the C ABI and not
a bad argument.  Each call runs in a process whose address space leaves no room for its row groups (no GPU)."""

import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CALLS = ["decode", "partial", "tree", "append", "write", "rope", "read", "prefill", "mass", "splits", "plan_write", "plan_decode",
         "plan_append"]


def child(name):
    import resource
    import numpy as np
    from paged_kv_cache_235_gb300 import binding as B
    FAKE = 1 << 20
    n = 8_000_000
    rs, rp = np.zeros(n, np.int32), np.zeros(n, np.int32)
    rp[1::2] = 5                                                 # no two rows in one group: 128 MB of them
    c = B.Cache("bf16", 8, 2, FAKE, FAKE, num_pages=64)
    segs = [B.Seg(1000, page_table=FAKE)]
    sc, plan = B.Scratch(FAKE, FAKE, n, 32), B.Plan()

    class Tensor:
        """A tensor's shape and address without the tensor."""
        is_contiguous = staticmethod(lambda: True)
        data_ptr = staticmethod(lambda: FAKE)

        def __init__(self, *shape):
            self.shape = shape
    table, mass = Tensor(1000, 64), Tensor(1, 2, 1024)
    calls = {
        "decode": lambda: B.tfpa_decode(c, segs, FAKE, rs, rp, 0.1, sc, FAKE, None, stream=0),
        "partial": lambda: B.tfpa_decode_partial(c, segs, FAKE, rs, rp, 0.1, sc, stream=0),
        "tree": lambda: B.tfpa_decode_tree(c, segs, FAKE, rs, rp, FAKE, 0.1, sc, FAKE, None, stream=0),
        "append": lambda: B.tfpa_decode_append(c, segs, FAKE, FAKE, FAKE, rs, rp, 0.1, sc, FAKE, None, stream=0),
        "write": lambda: B.tfpa_write_kv(c, segs, FAKE, FAKE, rs, rp, stream=0),
        "rope": lambda: B.tfpa_write_kv_rope(c, segs, FAKE, FAKE, rs, rp, table, table, stream=0),
        "read": lambda: B.tfpa_read_kv(c, segs, FAKE, FAKE, rs, rp, stream=0),
        "prefill": lambda: B.tfpa_prefill(c, segs, FAKE, rs, rp, 0.1, FAKE, None, stream=0),
        "mass": lambda: B.tfpa_key_mass(c, segs, FAKE, FAKE, rs, rp, 0.1, mass, stream=0),
        "splits": lambda: B.tfpa_row_splits(c, segs, rs, rp),
        "plan_write": lambda: plan.write_kv(c, segs, FAKE, FAKE, rs, rp),
        "plan_decode": lambda: plan.decode(c, segs, FAKE, rs, rp, 0.1, sc, FAKE, None),
        "plan_append": lambda: plan.decode_append(c, segs, FAKE, FAKE, FAKE, rs, rp, 0.1, sc, FAKE, None),
    }
    room = 2 * n * 4 if name in ("splits",) else 0                # the call's own result
    with open("/proc/self/status") as f:
        size = next(int(x.split()[1]) for x in f if x.startswith("VmSize")) * 1024
    with B.record_launches() as rec:
        resource.setrlimit(resource.RLIMIT_AS, (size + room + (16 << 20), resource.RLIM_INFINITY))
        try:
            calls[name]()
            print("done")
        except B.TfpaError as e:
            print("code", e.code, len(rec), B.strerror(e.code))
        resource.setrlimit(resource.RLIMIT_AS, (resource.RLIM_INFINITY, resource.RLIM_INFINITY))
    assert len(plan) == 0


@pytest.mark.parametrize("name", CALLS)
def test_host_memory_that_runs_out_is_an_error_code(name):
    from paged_kv_cache_235_gb300 import binding as B
    r = subprocess.run([sys.executable, "-c", f"from tests.test_host_memory import child; child({name!r})"], cwd=ROOT, capture_output=True,
                       text=True, timeout=120, env=dict(os.environ, OPENBLAS_NUM_THREADS="1", OMP_NUM_THREADS="1"))
    assert r.returncode == 0, (r.returncode, r.stderr[-600:])
    assert r.stdout.split()[:3] == ["code", str(B.TFPA_ENOMEM), "0"], r.stdout
    assert "memory" in r.stdout
