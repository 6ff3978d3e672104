"""The tests of window rows, of the attention over them and of drafted steps
under the bounds-checked library (libcsa2_debug.so), as a child process of
tests/test_gpu_window_debug.py with CSA2_DEBUG=1: every row of a cache, of drafts
and of outputs and every slot that a kernel forms has to stay inside (no error
word of any call is set), and the results are the tests'."""
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

import pytest  # noqa: E402
import torch  # noqa: E402

import fp4_kv_cache_index_gb300 as C  # noqa: E402

words = []          # error words of all caches and chunks
make, chunk = C.Window.__init__, C.csa2_window_attn_prefill


def made(self, *args, **kw):
    make(self, *args, **kw)
    words.append(self.error)


def checked(*args, **kw):
    if kw.get("error") is None:
        kw["error"] = words[0]
    return chunk(*args, **kw)


if __name__ == "__main__":
    assert C.LIB_PATH.endswith("libcsa2_debug.so"), C.LIB_PATH
    words.append(torch.zeros(4, dtype=torch.int32, device="cuda"))
    C.Window.__init__, C.csa2_window_attn_prefill = made, checked
    files = ["test_gpu_window.py", "test_gpu_window_positions.py", "test_gpu_window_nan_block.py",
             "test_gpu_drafted_step.py"]
    rc = pytest.main(["-q", "-x", "-m", "gpu", "-p", "no:cacheprovider",
                      *[os.path.join(ROOT, "tests", f) for f in files]])
    assert rc == 0, rc
    seen = sorted({int(w[0]) for w in words})   # (a word is the first of four)
    assert len(words) > 50 and seen == [0], seen
    print("window layers: all cases clean")
