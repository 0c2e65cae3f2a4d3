"""Rules that the CUDA sources keep and that no run can show to be broken (a run that breaks one may hang): read from
the sources."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "two_level_sparse_quest_b200", "csrc")


def sources():
    for name in sorted(os.listdir(CSRC)):
        if name.endswith((".cu", ".cuh")):
            with open(os.path.join(CSRC, name)) as f:
                yield name, re.sub(r"//[^\n]*", "", f.read())


def test_aligned_cluster_barriers_converge_the_warp_first():
    """barrier.cluster.*.aligned is executed by whole warps; its callers come from loops over a share of the outputs
    and from predicated loads, so the warp is converged directly before each of them."""
    seen = 0
    for name, text in sources():
        for m in re.finditer(r'asm volatile\(\s*"barrier\.cluster\.[a-z.]*aligned;"', text):
            seen += 1
            assert re.search(r"__syncwarp\(\);\s*$", text[:m.start()]), (name, text[max(0, m.start() - 80):m.end()])
    assert seen >= 3


def block_after(text, head):
    """The braced block that follows the first `head`."""
    i = text.index("{", text.index(head) + len(head))
    depth = 0
    for j in range(i, len(text)):
        depth += (text[j] == "{") - (text[j] == "}")
        if depth == 0:
            return text[i:j + 1]
    raise AssertionError(head)


def test_matrix_instructions_follow_a_converged_warp():
    """mma.sync and movmatrix take whole warps.  Before them lie a branch that the lanes of one head take alone (the
    attention's new maximum), and the ids and the adds of a tile (the accumulated weights)."""
    text = dict(sources())
    moved = block_after(text["tls_kv4_attn.cu"], "__any_sync(0xffffffffu, top > kPShift + 1.f))")
    assert "if (mx > m[nt][e])" in moved and re.search(r"__syncwarp\(\);\s*}$", moved)
    weights = text["tls_weights.cu"]
    for head in ("int token_at(const WeightsArgs &a, int group, int j, int n)", "void add_weight(float *p, float v, bool on)",
                 "for (; tile < tiles; tile += step)"):  # no branch of single lanes at all
        assert not re.search(r"\bif\s*\(", block_after(weights, head)), head


def test_a_copy_that_was_given_up_on_is_waited_for_again():
    """The attention's wait for a bulk copy has a limit.  Past it the kernel still waits, with the same limit, for the
    copy in flight before the ring is used for something else and the CTA's shared memory goes to another one."""
    text = dict(sources())["tls_kv4_attn.cu"]
    gave_up = block_after(text, "if (!__all_sync(0xffffffffu, arrived))")
    assert "atomicOr(a.err, kErrAttnWait)" in gave_up and "mbarrier_wait(&s_full[warp][st], phase)" in gave_up


def test_every_launcher_has_a_caller():
    """Each host launcher that a header declares is defined once and called."""
    names, text = set(), dict(sources())
    for name in sorted(os.listdir(CSRC)):
        if name.endswith(".h"):
            with open(os.path.join(CSRC, name)) as f:
                names |= set(re.findall(r"cudaError_t (launch_\w+)\([^;{]*\);", f.read()))  # declared, not defined
    assert len(names) > 10
    for n in sorted(names):
        seen = sum(len(re.findall(rf"\b{n}\(", t)) for t in text.values())
        defined = sum(len(re.findall(rf"cudaError_t {n}\(", t)) for t in text.values())
        assert seen > defined == 1, n
