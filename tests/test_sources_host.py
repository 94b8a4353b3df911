"""Rules that the kernels' sources keep and that no run of them shows reliably (no GPU)."""
import glob
import os
import re

from two_stage_kv_snapkv_gb300 import build_lib


def _sources():
    for path in sorted(glob.glob(os.path.join(build_lib.CSRC, "*.cu"))):
        with open(path) as f:
            yield os.path.basename(path), re.sub(r"//[^\n]*", "", f.read())


def test_barriers_are_fenced_by_the_threads_that_initialise_them():
    # fence.mbarrier_init orders the executing thread's own mbarrier.init before the copies
    # that complete on it: between an init and its fence no branch may change the threads
    seen = 0
    for name, text in _sources():
        for m in re.finditer(r"\bmbar_init\(", text):
            fence = text.find("fence_mbar_init();", m.end())
            line = text.count("\n", 0, m.start()) + 1
            assert fence >= 0, f"{name}:{line}: no fence behind the initialisation"
            between = text[m.end():fence]
            assert not re.search(r"\bif \(|\breturn\b|__global__", between), f"{name}:{line}: fenced by other threads"
            seen += 1
    assert seen > 10


def test_products_given_up_are_waited_for_before_their_memory_is_freed():
    # after a timeout a kernel that issues products between waits may hold one that no barrier
    # phase counts: only a commit made behind the last one tells when all are done
    for name, text in _sources():
        if name not in ("rkv_attend.cu", "rkv_accum.cu"):
            continue
        stop = text.index("if (abort_flag) {")
        free = text.index("tmem_dealloc(", stop)
        branch = text[stop:free]
        commit = branch.find("tc_commit_if(elect_lane(), &")
        assert commit >= 0, f"{name}: no commit behind the last product"
        bar = re.match(r"tc_commit_if\(elect_lane\(\), &([\w.]+)\)", branch[commit:]).group(1)
        assert f"mbar_wait(&{bar}, 0)" in branch[commit:], f"{name}: the commit is not waited for"
        assert text.count(f"mbar_init(&{bar}, 1)") == 1
