"""select_blocks refuses an output that overlaps what it reads, on the host before any CUDA call."""
import ctypes

from paged_kv_cache_230_gb300 import build


def test_tables_over_the_inputs():
    build.build()
    from paged_kv_cache_230_gb300 import pagedattn as pa
    far = lambda i, off=0: ctypes.c_void_p(0x10000000 * (i + 1) + off)  # noqa: E731

    def call(tables, S=3, Hkv=2, n=4, maxB=10):
        return pa.lib.pa_select_blocks(tables, far(1), n, far(2), far(3), maxB, far(4), S, Hkv, 16, 1, 1, None)

    scores, table, written = 3 * 2 * 10 * 4, 3 * 10 * 4, 3 * 2 * 4 * 4  # bytes
    for base, size in ((2, scores), (3, table)):
        assert call(far(base)) == -1 and call(far(base, size - 4)) == -1 and call(far(base, 4 - written)) == -1
