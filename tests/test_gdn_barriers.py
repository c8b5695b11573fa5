"""The named barriers of gdn_train's and gdn_backward's chains, on the CPU: every
order in which the warps of a tile can run is walked through, with the warps'
barrier calls as they stand in the source.

A named barrier counts contributions, not warps: one that contributes a second
time before the others have contributed at all stands in for a warp that is not
there yet, and the barrier opens early.  No order may allow that, and every order
must let all warps reach their end."""
import os
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "delta_rule_memory_gb300", "csrc", "gdn_train.cu")
CALL = re.compile(r"\b(meet|arrive)\((all|read|ready), 32 \* \(M \+ H\)\)")


def block(text, start):
    """The brace block that opens at or behind `start`."""
    at = text.index("{", start)
    depth = 0
    for i in range(at, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[at:i + 1]
    raise ValueError("unbalanced braces")


def calls(text):
    """(kind, barrier, whether only where a chunk follows), in order; of the two forms of an `if constexpr`, the first."""
    text = re.sub(r"//[^\n]*", "", text)
    while "if constexpr" in text:
        at = text.index("if constexpr")
        first = block(text, at)
        end = text.index(first, at) + len(first)
        other = re.match(r"\s*else\s*", text[end:])
        if other:
            second = block(text, end)
            assert calls(first) == calls(second)
            end = text.index(second, end) + len(second)
        text = text[:at] + first[1:-1] + text[end:]
    out = []
    for m in CALL.finditer(text):
        line = text[text.rfind("\n", 0, m.start()):m.start()]
        out.append((m[1], m[2], "c + 1 < n" in line))
    return out


def programs(kernel, chunks):
    """What a main and a helping warp call, over all chunks."""
    text = open(SOURCE).read()
    body = block(text, text.index(")", text.index(f"gdn_{kernel}(const Gdn a")))
    loops = [m.start() for m in re.finditer(r"for \(int c = (0; c < n; \+\+c|n - 1; c >= 0; --c)\) \{", body)]
    assert len(loops) == 2
    out = []
    for i, at in enumerate(loops):
        loop = calls(block(body, at))
        before = calls(body[body.index("if (me.role < M)"):at]) if i == 0 else []
        ops = [(k, b) for k, b, _ in before]
        for c in range(chunks):
            ops += [(k, b) for k, b, more in loop if not more or c + 1 < chunks]
        out.append(tuple(ops))
    return out


def walk(main, helper, M, H):
    """Every reachable state: of each kind of warps the sorted (calls done, waiting), and of each barrier who has contributed."""
    kinds = (main, helper)
    barriers = sorted({b for ops in kinds for _, b in ops})
    start = ((((0, None),) * M, ((0, None),) * H), tuple(() for _ in barriers))
    # a warp: (calls done, the barrier that it waits at or None); a barrier: sorted contributors as (kind, calls done then)
    seen, todo = {start}, [start]
    while todo:
        warps, inside = state = todo.pop()
        moved = False
        for kind, ops in enumerate(kinds):
            for i, (pc, waits) in enumerate(warps[kind]):
                if waits is not None or pc == len(ops) or (i and warps[kind][i - 1] == (pc, waits)):
                    continue
                moved = True
                what, name = ops[pc]
                b = barriers.index(name)
                # since the barrier last opened, a warp of this kind that stands here must not have contributed yet: all
                # its own earlier calls of the barrier lie in phases that are over
                mine = sum(o[1] == name for o in ops[:pc])
                if any(k == kind and before < mine for k, before in inside[b]):
                    return f"{'main' if kind == 0 else 'helping'} warp contributes again to a phase of `{name}`"
                here = inside[b] + ((kind, mine),)
                rows = [list(w) for w in warps]
                rows[kind][i] = (pc + 1, name if what == "meet" else None)
                left = list(inside)
                if len(here) == M + H:
                    rows = [[(p, None if w == name else w) for p, w in r] for r in rows]
                    here = ()
                left[b] = tuple(sorted(here))
                key = lambda w: (w[0], w[1] or "")  # noqa: E731
                new = (tuple(tuple(sorted(r, key=key)) for r in rows), tuple(left))
                if new not in seen:
                    seen.add(new)
                    todo.append(new)
        if not moved and any(pc < len(ops) or w for kind, ops in enumerate(kinds) for pc, w in warps[kind]):
            return f"no warp can go on: {state}"
    return None


@pytest.mark.parametrize("kernel", ["chain", "chain_back"])
@pytest.mark.parametrize("M,H", [(2, 1), (4, 2), (4, 4)])
def test_no_warp_stands_in_for_another(kernel, M, H):
    main, helper = programs(kernel, 3)
    assert {b for _, b in main} == {b for _, b in helper} and len(main) >= 6
    assert walk(main, helper, M, H) is None


def test_the_walk_sees_a_double_contribution():
    """A helping warp that is let past a barrier by warps that have yet to meet the one before."""
    main = (("arrive", "read"), ("meet", "all"), ("meet", "all"))
    helper = (("arrive", "all"), ("meet", "read"), ("meet", "all"))
    assert "helping warp contributes again" in walk(main, helper, 4, 4)
    assert walk((main[1], main[0], main[2]), helper, 4, 4) is None


def test_the_walk_sees_a_deadlock():
    assert "no warp" in walk((("meet", "all"), ("meet", "read")), (("meet", "read"), ("meet", "all")), 2, 1)
