"""Hand-overs inside the sampling kernel, read from its source: what one thread
writes for another is behind a barrier that orders it.  (None of them can be
provoked reliably on a GPU.)
"""
import os
import re

SOURCE = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "lossless_bit_weight_w12_gb300", "csrc",
                      "kernels_sample.cu")


def text():
    return re.sub(r"//[^\n]*", "", open(SOURCE).read())


def body(name):
    """The body of the function `name`."""
    s = text()
    at = s.index("{", re.search(r"\b%s\([^;{]*\{" % name, s).start())
    depth = 0
    for i in range(at, len(s)):
        depth += {"{": 1, "}": -1}.get(s[i], 0)
        if depth == 0:
            return s[at:i + 1]
    raise AssertionError(name)


def test_a_drawn_token_is_stored_before_the_row_is_counted():
    """Any thread of the cluster may store the token.  Counting the row for the
    acceptance has to be ordered after that store: by the storing thread itself,
    with a fence, or behind a barrier that releases what its warp wrote (a fence
    in CTA 0 orders only what CTA 0 has seen)."""
    kernel = body("sample_kernel")
    between = kernel[kernel.index("a.tokens[r] = token"):kernel.index("atomicAdd(a.counter")]
    by_itself = re.search(r"if \(writer\) \{\s*__threadfence\(\);\s*sh\.last = $", between)
    call = re.search(r"\b(sync_\w+)\((.*)\);", between)
    released = "cl.sync()" in between
    if call and not by_itself:
        arrive = body(call.group(1))
        released = "arrive.release" in arrive and (
            "arrive.relaxed" not in arrive or "writer" in call.group(2) and "__any_sync" in call.group(2))
    assert by_itself or released
    # the CTA of the storing thread goes on: its flag is reset in every CTA, and read behind a barrier
    if by_itself:
        assert kernel.index("if (tid == 0) sh.last = 0;") < kernel.index("cluster_started()")
        rest = kernel[kernel.index("atomicAdd(a.counter"):]
        assert rest.index("__syncthreads()") < rest.index("if (!sh.last) return;") < rest.index("__threadfence()")
        assert "me != 0" not in rest[:rest.index("a.accept_len[q]")] and "me != 0" not in between


def test_the_count_of_gathered_tokens_is_read_before_its_reset():
    """In window_threshold all threads read list_n and branch on it, and thread
    0 resets it for the next turn: a warp that read late would see 0, leave the
    loop and meet other barriers than its CTA.  Walks the function's statements
    in their order, the loop's twice: between a read and the next write of
    list_n there is a barrier."""
    b = body("window_threshold")
    loop = b.index("while (m > 128u)")
    start = b.index("{", loop)
    depth, end = 0, start
    for end in range(start, len(b)):
        depth += {"{": 1, "}": -1}.get(b[end], 0)
        if depth == 0:
            break
    run = b[:end] + b[start:end] + b[end:]
    events = re.findall(r"__syncthreads\(\)|boundary_bin\(|m = sh\.list_n|sh\.list_n = 0u|atomicAdd\(&sh\.list_n", run)
    assert events.count("m = sh.list_n") == 3 and events.count("sh.list_n = 0u") == 3
    read = False
    for e in events:
        if e in ("__syncthreads()", "boundary_bin("):  # (boundary_bin begins and ends with one)
            read = False
        elif e == "m = sh.list_n":
            read = True
        else:
            assert not read, e
    bin_body = body("boundary_bin")
    assert bin_body.lstrip("{ \n").split(";")[1].strip() == "__syncthreads()"


def test_all_ctas_have_started_before_the_first_remote_access():
    """Another CTA's shared memory may be touched only once that CTA has
    started: behind a barrier of the whole cluster."""
    kernel = body("sample_kernel")
    first = kernel.index("map_shared_rank")
    barriers = [kernel.find(x) for x in ("cl.sync()", "sync_sums()", "sync_written(", "cluster_started()")]
    barriers = [x for x in barriers if x >= 0]
    assert barriers and min(barriers) < first
    assert kernel.index("cluster_here()") < kernel.index("cluster_started()") < first
    assert "barrier.cluster.arrive" in body("cluster_here") and "barrier.cluster.wait" in body("cluster_started")
