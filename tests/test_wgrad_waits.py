"""The waits of wgrad_stream_kernel that are counted by hand, against the compiler's listing of it (CPU only; hipcc needed).

While a block is multiplied, copies of later blocks into LDS are under way.  The barrier before the next block waits for all but
the youngest N loads and stores of a wave: this block's 4 copies of rows, its scale bytes' loads and, behind a finished tile,
the tile's stores.  Were one of those merged with another or left out by a compiler, N would reach back to a copy of the next
block's columns, and the block could be read before it is there.  So on every path that leads to such a barrier, the
youngest N accesses must hold no copies but the 4 of this block."""
import os
import re
import subprocess

import pytest

from fine_grained_quantization_amd import build

NAMES = {"bf16": "Lb0ELb0E", "bf16, added": "Lb0ELb1E", "fp32": "Lb1ELb0E", "fp32, added": "Lb1ELb1E"}
COUNTED = re.compile(r"s_waitcnt vmcnt\((\d+)\) lgkmcnt\(0\)$")
OWN_COPIES = 4


@pytest.fixture(scope="module")
def listing(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("listing") / "wgrad.s")
    cmd = [build.HIPCC, *build.FLAGS, "--cuda-device-only", "-S", os.path.join(build.CSRC, "fp8q_wgrad.hip"), "-o", out]
    subprocess.run(cmd, check=True, capture_output=True)
    with open(out) as f:
        return f.read().splitlines()


def kernel(listing, name):
    """A kernel's lines, as (label or None, instruction)."""
    at = next(i for i, l in enumerate(listing) if re.match(r"_ZN\w*wgrad_stream_kernelI" + name + r"\w*:", l))
    body = []
    for l in listing[at + 1:]:
        if l.startswith(".Lfunc_end"):
            return body
        l = l.split(";")[0].strip()
        label = re.match(r"(\.LBB\w+):", l)
        if label:
            body.append((label.group(1), ""))
        elif l and not l.startswith("."):
            body.append((None, l))
    raise AssertionError("the kernel's end is missing")


def before(body):
    """For each line, those that may run right before it."""
    at = {label: i for i, (label, _) in enumerate(body) if label}
    prev = [[] for _ in body]
    for i, (_, op) in enumerate(body):
        jump = re.match(r"s_c?branch\S*\s+(\.LBB\w+)", op)
        if jump:
            prev[at[jump.group(1)]].append(i)
        if i + 1 < len(body) and not op.startswith(("s_branch", "s_endpgm")):
            prev[i + 1].append(i)
    return prev


def short_paths(body):
    """Counted barriers, and the paths to them on which the youngest N accesses hold a fifth copy."""
    prev, found, bad = before(body), [], []
    for i, (_, op) in enumerate(body):
        n = COUNTED.match(op)
        if not n or body[i + 1][1] != "s_barrier":
            continue
        n = int(n.group(1))
        own = OWN_COPIES if found else 2 * OWN_COPIES  # (the first one, before the loop: the second block's rows and columns)
        found.append(n)
        stores = n - OWN_COPIES > 8  # this wait counts a tile's stores: it is only reached behind them
        todo, seen = [(i, 0, 0, False)], set()
        while todo:
            j, count, copies, stored = todo.pop()
            for k in prev[j]:
                op = body[k][1]
                state = (k, count, copies, stored)
                if re.match(r"(buffer|global|flat|scratch)_", op):
                    copy = op.endswith("lds")
                    if copy and copies == own and (stored or not stores):
                        bad.append((n, i, k, count))
                        continue
                    if count + 1 >= n or (copy and copies == own):
                        continue  # (enough, or a path that the wait is not reached on)
                    state = (k, count + 1, copies + copy, stored or "_store" in op)
                if state not in seen:
                    seen.add(state)
                    todo.append(state)
    return found, bad


@pytest.mark.parametrize("name", NAMES.values(), ids=NAMES)
def test_counted_waits(listing, name):
    body = kernel(listing, name)
    found, bad = short_paths(body)
    scales, stores = (3, 32) if name.startswith("Lb1") else (2, 16)
    # one before the loop, and in the loop's two blocks one without and one with a tile's stores
    assert sorted(found) == sorted([8] + 2 * [OWN_COPIES + scales, OWN_COPIES + scales + stores])
    assert not bad, bad[:5]
    assert all(not op.startswith("scratch_") for _, op in body)  # (a reload would wait for all copies)


@pytest.mark.parametrize("name", NAMES.values(), ids=NAMES)
def test_a_missing_access_is_noticed(listing, name):
    """The listing with one scale load of the loop taken out, or one store.  (Where old results are added, their loads are
    between the copies and the wait as well, and a store less is no harm.)"""
    body = kernel(listing, name)
    loop = next(i for i, (_, op) in enumerate(body) if COUNTED.match(op)) + 1
    scales = [i for i, (_, op) in enumerate(body) if i > loop and re.match(r"buffer_load_dword(x2)? ", op)]
    stores = [i for i, (_, op) in enumerate(body) if i > loop and op.startswith("buffer_store")]
    assert len(scales) == (6 if name.startswith("Lb1") else 4) and len(stores) == (64 if name.startswith("Lb1") else 32)
    for gone in (scales[0], scales[-1], *([] if name.endswith("Lb1E") else [stores[0], stores[-1]])):
        assert short_paths(body[:gone] + body[gone + 1:])[1], body[gone]
