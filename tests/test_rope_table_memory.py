"""w12_rope_table allocates nothing: it works, and throws nothing across the C
entry, where no memory is left."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = """
import resource
import numpy as np
from lossless_bit_weight_w12_gb300 import w12
L = w12.lib()
rot = 1 << 24
table = np.ones((1, rot), dtype=np.float32)
small = w12.rope_table(3, 1000, 1e4, w12.ROPE_SCALE_YARN, factor=4.0, original=64.0)
pages = int(open("/proc/self/statm").read().split()[0])
room = pages * resource.getpagesize() + (16 << 20)
resource.setrlimit(resource.RLIMIT_AS, (room, room))
try:
    np.ones(rot // 2)
    raise SystemExit(3)  # the limit does not hold
except MemoryError:
    pass
st = L.w12_rope_table(1, rot, 1e4, None, w12._np_ptr(table))
assert st == w12.OK, st
assert (table[0, :rot // 2] == 1).all() and (table[0, rot // 2:] == 0).all()  # position 0
again = w12.rope_table(3, 1000, 1e4, w12.ROPE_SCALE_YARN, factor=4.0, original=64.0)
assert (small == again).all()
"""


def test_no_memory_left():
    env = dict(os.environ, OMP_NUM_THREADS="1", OPENBLAS_NUM_THREADS="1", PYTHONPATH=ROOT)
    p = subprocess.run([sys.executable, "-c", CHILD], cwd=ROOT, env=env, capture_output=True, text=True, timeout=120)
    assert p.returncode == 0, (p.returncode, p.stderr[-2000:])
