"""What sd_logprobs reads, shown in its source: a read that should not be would fault, not fail."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_a_row_that_is_not_scored_is_not_read():
    """The kernel looks at the row's token, and leaves, before its first load of the row."""
    with open(os.path.join(ROOT, "verify_step_b200", "csrc", "logprobs.cu")) as f:
        src = re.sub(r"//[^\n]*", "", f.read())
    body = src[src.index("chunk_kernel(const"):src.index("merge_kernel(const")]
    leaves = re.search(r"if \(!scored\([^;]*\)\) return;", body).start()
    reads = [m.start() for m in re.finditer(r"\bload_tile<|\bz\[", body)]
    assert reads and leaves < min(reads)
