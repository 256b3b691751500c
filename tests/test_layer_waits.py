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
    assert "mbarrier.try_wait" in wait and re.search(r"bool (\w+) = __all_sync\(0xffffffffu, \w+\);.*return \1;\s*\}$", wait, re.S)
    assert wait.count("return") == 1


def kernels():
    text = source()
    return [function(text, r"\bgemm_kernel\("), function(text, r"\bnarrow_backward_kernel\(")]


def test_blocks_stay_until_free_stages_are_reported():
    """The multiplying warp's reports of free stages arrive at a barrier of the block after its last wait for it: the
    copying warp of each kernel waits once more for every stage."""
    for k in kernels():
        assert re.search(r"Ring last = r;\s*for \(int (\w) = 0; \1 < g\.stages && ok; \+\+\1, last\.next\(g\.stages\)\) "
                         r"ok = warp_waits<\w+>\(empty \+ 8 \* last\.stage", k)


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


def test_a_pair_gives_up_together():
    """The copies of a pair's second block are counted by the first one's barriers. So the second block cannot wait for
    them: a block that gives up tells the other, and the first one waits for the copies of both, however many
    each of them had issued, before either leaves."""
    assert "st.relaxed.cluster.shared::cluster" in function(source(), r"bool warp_waits\(")
    k = kernels()[0]
    drain = k[k.rindex("if (abort_flag != 0) {"):k.index("tcgen05.dealloc")]
    assert k[:k.rindex("if (abort_flag != 0) {")].rstrip().endswith("if (kPair) cluster_sync();")
    assert drain.index("arrive_expect(") < drain.index("count_copied(") < drain.index("wait_parity(full") < drain.index("if (kPair) cluster_sync();")


def left_waiting(stages, first, second, mended=True):
    """Model of the first block's barriers: two copies and one announcement a stage and lap, the blocks ending after
    `first` and `second` stages. Returns the laps of stages that were issued and never counted as complete."""
    tx, announced = {}, {}
    for c in range(first):                       # the first block announces both copies, and its own arrives
        announced[c] = 2
        tx[c] = tx.get(c, 0) + 1
    for c in range(second):
        tx[c] = tx.get(c, 0) + 1
    most = max(first, second)
    if mended:
        for c in range(first, most):
            announced[c] = 1
        for c in range(second, most):
            tx[c] = tx.get(c, 0) + 1
    return [c for c in range(max(0, most - stages), most) if announced.get(c) != tx.get(c)]


def test_copies_in_flight_of_a_pair_are_all_counted():
    for stages in (1, 4, 5):
        for first in range(12):
            for second in range(max(0, first - stages), first + stages + 1):
                assert left_waiting(stages, first, second) == []
                assert (left_waiting(stages, first, second, mended=False) == []) == (first == second)
