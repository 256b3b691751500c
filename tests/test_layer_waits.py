"""The waits of the layers' kernels: none is unbounded, and a block that gives one up ends in order."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "multiresolution_hash_grid_b200", "csrc")


def source():
    """hg_linear.cuh without its comments."""
    with open(os.path.join(CSRC, "hg_linear.cuh")) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def function(text, head):
    """The body of the function whose signature `head` matches."""
    at = text.index("{", re.search(head, text).end())
    depth, end = 0, at
    while True:
        depth += (text[end] == "{") - (text[end] == "}")
        end += 1
        if depth == 0:
            return text[at:end]


def test_waits_are_votes_of_whole_warps():
    """A warp goes on, or gives up, as a whole: lanes that polled a barrier for themselves could part (one gives up
    where another sees the phase flip) and then stop at different meetings for good."""
    text = source()
    assert text.count("mbarrier.try_wait") == 1 and "test_wait" not in text
    wait = function(text, r"bool warp_waits\(")
    assert "mbarrier.try_wait" in wait and re.search(r"__all_sync\(0xffffffffu, \w+\);\s*if \(!\w+\) \*abort_flag = 1;\s*return \w+;\s*\}$", wait)


def kernels():
    text = source()
    return [function(text, r"\bgemm_kernel\("), function(text, r"\bnarrow_backward_kernel\(")]


def test_blocks_stay_until_free_stages_are_reported():
    """The multiplying warp's reports of free stages arrive at a barrier of the block after its last wait for it: the
    copying warp of each kernel waits once more for every stage."""
    for k in kernels():
        assert re.search(r"Ring last = r;\s*for \(int (\w) = 0; \1 < g\.stages && ok; \+\+\1, last\.next\(g\.stages\)\) "
                         r"ok = warp_waits\(empty \+ 8 \* last\.stage", k)


def test_tensor_memory_is_freed_by_a_whole_warp():
    """The warp that frees it meets after a branch that one lane takes alone."""
    for k in kernels():
        tail = k[:k.index("tcgen05.dealloc")]
        assert re.search(r"__syncwarp\(\);\s*if \(warp == 0\)[^;]*$", tail)


def test_a_block_that_gave_up_ends_after_its_copies_and_products():
    """Whichever role gave up, the copying and the multiplying warp wait for what they issued, after all roles have
    ended and before tensor memory is freed."""
    for k in kernels():
        tail = k[:k.index("tcgen05.dealloc")]
        tail = tail[tail.rindex("if (abort_flag != 0) {"):]
        assert "copies_issued" in tail and "commit(drain)" in tail and "wait_parity(drain, 0)" in tail and "__syncthreads();" in tail
        assert k.count("wait_parity(drain, 0)") == 1 and "__syncthreads();" in k[:k.rindex("if (abort_flag != 0) {")][-60:]
