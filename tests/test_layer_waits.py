"""The waits of the layers' kernels: none is unbounded, and a block that gives one up ends in order."""
import os
import re

import pytest

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


SHAPES = [(16, 2048, 1024), (333, 77, 130), (2000, 64, 96), (50000, 64, 64), (40, 4096, 264),  # over clusters, odd, plain, kept weights
          (19100, 512, 160), (5000, 1600, 1030), (9700, 1000, 300),                            # pairs, also gathering
          (90001, 64, 64), (20000, 128, 128), (30000, 27, 31)]                                 # one-pass backward


def calls(hg, torch, shape, y32):
    """One forward and one backward call of a layer as a function that returns their outputs and their status words."""
    N, K, M = shape
    gen = torch.Generator(device="cuda").manual_seed(N + K)
    layer = hg.Linear(K, M, activation=hg.HASHGRID_ACT_SILU if y32 else hg.HASHGRID_ACT_RELU)
    x, w, dy, z = (torch.randn(*s, device="cuda", generator=gen).bfloat16() for s in ((N, K), (M, K), (N, M), (N, M)))
    kind = torch.float32 if y32 else torch.bfloat16
    out = [torch.empty(N, M, device="cuda", dtype=kind), torch.empty(N, K, device="cuda", dtype=kind),
           torch.empty(M, K, device="cuda"), torch.empty(M, device="cuda")]
    work, status = layer.workspace(N, "cuda"), torch.zeros(8, dtype=torch.int32, device="cuda")

    def run():
        status.zero_()
        for t in out:
            t.fill_(7.0)
        layer.forward(x, w, y=out[0], workspace=work, device_status=status[:4])
        layer.backward(dy, x, w, z=z, dL_dx=out[1], dL_dw=out[2], dL_db=out[3], workspace=work, device_status=status[4:])
        torch.cuda.synchronize()
        return [t.clone() for t in out], status[::4].tolist()
    return run


@pytest.mark.gpu
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_waits_that_run_out(shape):
    """With a limit of no polls each call gives up and says so; with few, it gives up or is right; afterwards it is right."""
    import torch

    import multiresolution_hash_grid_b200 as hg
    for y32 in (False, True):
        run = calls(hg, torch, shape, y32)
        want, status = run()
        assert status == [0, 0]
        try:
            for limit in (0, 1, 2, 3, 5, 9, 30, 0):
                hg.hashgrid_debug_wait_limit(limit)
                got, status = run()
                assert status == [1, 1] or limit > 0
                if status[0] == 0:
                    assert torch.equal(got[0], want[0])
                if status[1] == 0:
                    assert all(torch.equal(a, b) for a, b in zip(got[1:], want[1:]))
        finally:
            hg.hashgrid_debug_wait_limit()
        got, status = run()
        assert status == [0, 0] and all(torch.equal(a, b) for a, b in zip(got, want))


GIVE_UP = r"""
import os, time, torch, multiresolution_hash_grid_b200 as hg
from tests.test_layer_waits import SHAPES, calls
assert "checked" in hg.hashgrid_version()
seen = set()
for shape in SHAPES:
    for y32 in (False, True):
        run = calls(hg, torch, shape, y32)
        want, status = run()
        assert status == [0, 0], shape
        for role in (1, 2, 3, 4):
            for nth in (1, 2, 3, 6):
                for parity in (0, 1, 2):
                    os.environ["HASHGRID_CHECK_GIVE_UP"] = "%d,%d,%d" % (role, nth, parity)
                    t = time.time()
                    got, status = run()
                    assert time.time() - t < 20, (shape, role, nth, parity)
                    assert role == 4 or nth > 1 or parity != 2 or status == [1, 1], (shape, role, status)
                    if status[0] == 0:
                        assert torch.equal(got[0], want[0])
                    else:
                        seen.add((role, nth))
                    if status[1] == 0:
                        assert all(torch.equal(a, b) for a, b in zip(got[1:], want[1:]))
                    else:
                        seen.add((role, nth))
        del os.environ["HASHGRID_CHECK_GIVE_UP"]
        got, status = run()
        assert status == [0, 0] and all(torch.equal(a, b) for a, b in zip(got, want)), shape
    print(shape, flush=True)
assert len(seen) == 16, seen
print("ok")
"""


@pytest.mark.gpu
@pytest.mark.timeout(900)
def test_any_role_gives_up_at_any_time():
    """The copying, the multiplying, the writing and the dz warps in turn, at their first and at later waits, with
    copies and products under way, in the blocks of one side of a pair or in all: each call returns and says so."""
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", GIVE_UP], cwd=root, env=dict(os.environ, HASHGRID_CHECKED="1"), capture_output=True,
                       text=True, timeout=800)
    assert r.returncode == 0 and r.stdout.endswith("ok\n"), r.stdout[-2000:] + r.stderr[-2000:]


@pytest.mark.gpu
def test_a_call_that_gave_up_without_a_status_word_is_reported():
    """By the next call, which does nothing else, or by the status call; once; also out of a captured graph."""
    import torch

    import multiresolution_hash_grid_b200 as hg
    layer = hg.Linear(64, 96)
    gen = torch.Generator(device="cuda").manual_seed(3)
    x, w = (torch.randn(*s, device="cuda", generator=gen).bfloat16() for s in ((500, 64), (96, 64)))
    want = layer.forward(x, w)
    hg.hashgrid_linear_status()
    y, seven = torch.empty_like(want), torch.full_like(want, 7.0)

    def give_up():
        try:
            hg.hashgrid_debug_wait_limit(0)
            layer.forward(x, w, y=y)
        finally:
            hg.hashgrid_debug_wait_limit()

    def refused(call):
        with pytest.raises(hg.HashGridError, match="incomplete") as e:
            call()
        assert e.value.code == hg.HASHGRID_ERR_TIMEOUT
    for call in (lambda: layer.forward(x, w, y=seven), lambda: layer.backward(want, x, w), hg.hashgrid_linear_status):
        give_up()
        torch.cuda.synchronize()
        refused(call)
        torch.cuda.synchronize()
        assert bool((seven == 7.0).all())
        assert torch.equal(layer.forward(x, w), want)
        hg.hashgrid_linear_status()
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    hg.hashgrid_debug_wait_limit(0)
    layer.forward(x, w, y=y, device_status=status)
    hg.hashgrid_debug_wait_limit()
    torch.cuda.synchronize()
    assert int(status[0]) == 1
    hg.hashgrid_linear_status()                        # a call with a status word of its own is not reported twice
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        give_up()
    torch.cuda.synchronize()
    hg.hashgrid_linear_status()
    g.replay()
    torch.cuda.synchronize()
    refused(hg.hashgrid_linear_status)


@pytest.mark.gpu
def test_the_first_call_of_a_process_may_be_captured():
    import subprocess
    import sys
    code = r"""
import torch, multiresolution_hash_grid_b200 as hg
x, w = torch.ones(300, 64, device="cuda").bfloat16(), torch.ones(96, 64, device="cuda").bfloat16()
y, layer, g = torch.zeros(300, 96, device="cuda").bfloat16(), hg.Linear(64, 96), torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    layer.forward(x, w, y=y)
g.replay()
torch.cuda.synchronize()
assert bool((y == 64).all())
hg.hashgrid_linear_status()
print("ok")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, env=dict(os.environ, HASHGRID_CHECKED="0"), capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "ok" in r.stdout, r.stdout + r.stderr


@pytest.mark.gpu
def test_asking_for_the_status_first_makes_no_context():
    """A process that has called no layer has nothing to report, and asking leaves the device alone."""
    import subprocess
    import sys
    code = r"""
import ctypes, multiresolution_hash_grid_b200 as hg
cu = ctypes.CDLL("libcuda.so.1")
hg.hashgrid_linear_status()
flags, active = ctypes.c_uint(), ctypes.c_int(7)
assert cu.cuInit(0) == 0 and cu.cuDevicePrimaryCtxGetState(0, ctypes.byref(flags), ctypes.byref(active)) == 0
assert active.value == 0, active.value
print("ok")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, env=dict(os.environ, HASHGRID_CHECKED="0"), capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "ok" in r.stdout, r.stdout + r.stderr


@pytest.mark.gpu
def test_calls_from_several_threads():
    """Handles, the wait limit's and the status words' state and the launch attributes are shared between threads."""
    import threading

    import torch

    import multiresolution_hash_grid_b200 as hg
    if hg.CHECKED:
        pytest.skip("the checked build is for one stream at a time")
    jobs = [calls(hg, torch, shape, y32) for shape in SHAPES for y32 in (False, True)]
    want = [run() for run in jobs]
    failed = []

    def work(k):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(5):
                got, status = jobs[k]()
                if status != [0, 0] or not all(torch.equal(a, b) for a, b in zip(got, want[k][0])):
                    failed.append(SHAPES[k // 2])
    threads = [threading.Thread(target=work, args=(k,)) for k in range(len(jobs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert failed == []
