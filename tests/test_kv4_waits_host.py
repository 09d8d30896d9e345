"""What the attention kernels wait for, read from their source (no GPU needed)."""
import os
import random
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "tensor_sharded_linear_gb300", "csrc")


def code(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def kernels():
    """(file, body) of every kernel that is launched before the one ahead of it has ended."""
    for name in sorted(os.listdir(CSRC)):
        if not name.endswith((".cu", ".cuh")) or name == "heads_sm103.cuh":
            continue
        for part in code(name).split("__global__")[1:]:
            if "wait_for_previous_kernel();" in part:
                yield name, part


def test_tensor_memory_is_taken_after_the_kernel_before_has_ended():
    """A CTA that held tensor memory while waiting could keep a CTA of that kernel from its own: neither would end."""
    seen = 0
    for name, body in kernels():
        at = body.find("tcgen05.alloc")
        if at >= 0:
            seen += 1
            assert body.find("wait_for_previous_kernel();") < at, name
    assert seen == 1


def test_warps_that_give_up_come_to_the_meetings_all_the_same():
    """A named barrier between warps has no time limit of its own: a warp that leaves a loop with such a meeting early
    has to come to the rest of them, or its partner waits there for good."""
    body = code("kv4_prompt.cuh")
    role = body[body.index("warp >= 8 && warp < 12"):body.index("warp == 12")]
    loop, after = role.split("while (!ok)")
    assert len(re.findall(r'"bar\.sync %0, 64;"', loop)) == 1 and len(re.findall(r'"bar\.(sync|red)', body)) == 2
    before, behind = loop.split("bar.sync")
    breaks = [re.findall(r"left = (s\.nb - i[^;]*);\s*break;", x) for x in (before, behind)]
    assert breaks == [["s.nb - i"], ["s.nb - i - 1"]]  # of this unit's, with and without this step's
    assert loop.count("break;") == 2
    assert re.search(r'for \(; left > 0; --left\) asm volatile\("bar\.sync %0, 64;" ::"r"\(1 \+ kv\) : "memory"\);\s*'
                     r"if \(!advance\(s\)\) break;\s*left = s\.nb;", after)
    assert not re.search(r'"bar\.(sync|red)', "".join(part for name, part in kernels() if name != "kv4_prompt.cuh"))


def meetings(units, fails, seed, stay=True):
    """Two warps over units of steps of wait, meeting, wait; a warp's wait may run out, or give up because another role
    raised the abort flag.  Interleaved at random; True if both come to an end."""
    rng = random.Random(seed)
    flag, arrived, generation = [False], [0], [0]

    def gives_up(key):
        return key in fails or (flag[0] and rng.random() < 0.5)  # (a wait may succeed though the flag is raised)

    def meet():
        arrived[0] += 1
        g = generation[0]
        if arrived[0] == 2:
            arrived[0] = 0
            generation[0] += 1
        while generation[0] == g:
            yield
        yield

    def warp(me):
        todo, ok, left, n = list(units), True, 0, 0
        while ok and todo:
            nb = todo.pop(0)
            for i in range(nb):
                yield
                if gives_up((me, n, 0)):
                    flag[0], ok, left = True, False, nb - i
                    break
                yield from meet()
                if gives_up((me, n, 1)):
                    flag[0], ok, left = True, False, nb - i - 1
                    break
                n += 1
        while stay and not ok:
            for _ in range(left):
                yield from meet()
            if not todo:
                break
            left = todo.pop(0)

    live = {i: warp(i) for i in (0, 1)}
    for _ in range(3000):
        if not live:
            return True
        if fails and rng.random() < 0.02:
            flag[0] = True
        i = rng.choice(sorted(live))
        try:
            next(live[i])
        except StopIteration:
            del live[i]
    return False


def test_meetings_end_however_the_warps_give_up():
    held = 0
    for seed in range(3000):
        rng = random.Random(seed)
        units = [rng.randrange(1, 5) for _ in range(rng.randrange(1, 4))]
        fails = {(rng.randrange(2), rng.randrange(sum(units)), rng.randrange(2)) for _ in range(rng.randrange(4))}
        assert meetings(units, fails, seed), seed
        held += not meetings(units, fails, seed, stay=False)
    assert held > 100  # warps that leave for good do hold their partners
